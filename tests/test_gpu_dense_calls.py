"""Calls of the dense layer at the edges of its arguments: arrays that overlap, row strides of a single row, outputs that
autograd has seen, layers of more than 2^32 weights."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def refused(call, *args):
    import qml_gradients_amd as hq
    with pytest.raises(hq.HqmlError) as e:
        call(*args)
    assert e.value.status == hq.HQML_ERR_ARG and "overlap" in str(e.value)


def test_outputs_that_overlap_an_argument_are_refused():
    """Workgroups write some rows of an output while others still read theirs."""
    import qml_gradients_amd as hq
    M, K, N = 12, 16, 16
    layer = hq.Dense(K, N, M, activation="tanh")
    buf = torch.randn(4 * M, K, device="cuda")
    x, w, bias, r = buf[:M], torch.randn(N, K, device="cuda"), torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda")
    before = buf.clone()
    refused(lambda: layer.forward(x, w, out=buf[1:M + 1]))              # a row on
    refused(lambda: layer.forward(buf[3:M + 3], w, out=buf[:M]))        # from behind
    both = torch.randn(M, K + N, device="cuda")
    refused(lambda: layer.forward(both[:, :K], w, out=both[:, K - 1:-1]))   # one column in common
    refused(lambda: layer.forward(x, w, both.view(-1)[K + N:K + 2 * N], out=both[:, :N]))   # the bias is a row of it
    refused(lambda: layer.forward(x, w, residual=buf[2 * M:3 * M], out=buf[2 * M + 1:3 * M + 1]))
    refused(lambda: layer.forward(x.clone(), w, residual=buf.view(-1, 2 * K)[:M, :K], out=buf[:M]))   # another row stride
    weights = torch.randn(M + N, K, device="cuda")
    refused(lambda: layer.forward(x, weights[M - 1:M - 1 + N], out=weights[:M]))
    y, z = layer.forward_train(x, w, bias, r)
    p = [t.data_ptr() for t in (x, w, z, r)]
    refused(hq.hqml_dense_forward, layer.handle, M, p[0], K, p[1], K, None, None, 0, y.data_ptr(), N, y.data_ptr() + 64)
    refused(hq.hqml_dense_backward, layer.handle, M, p[3], N, p[0], K, p[1], K, p[2], p[0], K, None, None)
    refused(hq.hqml_dense_backward, layer.handle, M, p[3], N, p[0], K, p[1], K, p[2], None, K, p[1], None)
    refused(hq.hqml_dense_backward, layer.handle, M, p[3], N, p[0], K, p[1], K, p[2], None, K, None, p[2] + 4)
    dw = torch.zeros(N, K, device="cuda")
    refused(hq.hqml_dense_backward, layer.handle, M, p[3], N, p[0], K, p[1], K, p[2], None, K, dw.data_ptr(),
            dw.data_ptr() + 8)
    torch.cuda.synchronize()
    assert torch.equal(buf, before) and not dw.any()


def test_outputs_beside_their_arguments_are_taken():
    """Columns of one array, rows that follow one another, a bias in the gap between output rows, the residual itself."""
    import qml_gradients_amd as hq
    M, K, N = 12, 16, 24
    layer = hq.Dense(K, N, M, activation="tanh")
    x, w, bias, r = (torch.randn(*s, device="cuda") for s in ((M, K), (N, K), (N,), (M, N)))
    want = layer.forward(x, w, bias, r)
    wide = torch.randn(M, K + 3 * N, device="cuda")
    wide[:, :K], wide[:, K:K + N], wide[3, -N:] = x, r, bias
    keep = wide.clone()
    got = layer.forward(wide[:, :K], w, wide[3, -N:], wide[:, K:K + N], out=wide[:, K + N:K + 2 * N])
    assert torch.equal(got, want)
    keep[:, K + N:K + 2 * N] = want
    assert torch.equal(wide, keep)
    rows = torch.zeros(2 * M, N, device="cuda")
    rows[:M] = r
    assert torch.equal(layer.forward(x, w, bias, rows[:M], out=rows[M:]), want)
    assert torch.equal(layer.forward(x, w, bias, rows[:M], out=rows[:M]), want)
    one = rows[M - 1:M].clone()   # one row's stride means nothing
    one.copy_(r[:1])
    assert torch.allclose(layer.forward(x[:1], w, bias, one, out=one), want[:1], atol=1e-5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["none", "tanh"])
def test_stride_of_a_single_row_means_nothing(act, dtype):
    """Of an array of one row any stride is as good as another, 2^30 elements (2^32 bytes) too."""
    import qml_gradients_amd as hq
    for M, K, N in ((1, 40, 24), (1, 300, 1), (7, 33, 1)):
        say(f"[gpu] dense {M} x {K} -> {N} {dtype} {act}")
        dt = torch.float32 if dtype == "fp32" else torch.bfloat16
        x, w, r, dy = (torch.randn(*s, device="cuda").to(dt) for s in ((M, K), (N, K), (M, N), (M, N)))
        layer = hq.Dense(K, N, M, dtype=dtype, activation=act)
        want, z = layer.forward_train(x, w, None, r)
        grads = layer.backward(dy, x, w, z)
        zp = None if z is None else z.data_ptr()
        for far in (1 << 20, 1 << 30, (1 << 30) + 8, 1 << 31, 1 << 40):
            lx, lw, ly = far if M == 1 else K, far if N == 1 else K, far if M == 1 else N
            y = torch.zeros_like(r)
            hq.hqml_dense_forward(layer.handle, M, x.data_ptr(), lx, w.data_ptr(), lw, None, r.data_ptr(), ly,
                                  y.data_ptr(), ly, zp)
            assert torch.equal(y, want)
            got = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(N, dtype=dt, device="cuda")
            hq.hqml_dense_backward(layer.handle, M, dy.data_ptr(), ly, x.data_ptr(), lx, w.data_ptr(), lw, zp,
                                   got[0].data_ptr(), lx, got[1].data_ptr(), got[2].data_ptr())
            assert all(torch.equal(a, b) for a, b in zip(got, grads)), far
        same = r[:1].clone()
        if M == 1:   # the residual itself, whatever the strides say
            hq.hqml_dense_forward(layer.handle, 1, x.data_ptr(), K, w.data_ptr(), K, None, same.data_ptr(), N,
                                  same.data_ptr(), N + 8, None)
            assert torch.equal(same, want)


def test_out_marks_its_array_changed():
    """A backward pass that saved the array from before the call has to refuse it."""
    import qml_gradients_amd as hq
    layer = hq.Dense(8, 6, 4)
    x, w, out = (torch.randn(*s, device="cuda") for s in ((4, 8), (6, 8), (4, 6)))
    a = torch.ones(4, 6, device="cuda", requires_grad=True)
    loss = (a * out).sum()
    layer.forward(x, w, out=out)
    with pytest.raises(RuntimeError):
        loss.backward()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_empty_batch_of_a_layer_of_2_to_the_32_weights(dtype):
    """Its dw is zeros like any other's."""
    import qml_gradients_amd as hq
    K = N = 1 << 16
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    layer = hq.Dense(K, N, 4, dtype=dtype)
    dw = torch.ones(N, K, dtype=layer.dtype, device="cuda")
    db = torch.ones(N, dtype=layer.dtype, device="cuda")
    hq.hqml_dense_backward(layer.handle, 0, None, N, None, K, None, K, None, None, K, dw.data_ptr(), db.data_ptr())
    assert not db.any() and int(torch.count_nonzero(dw[:2])) == 0 and int(torch.count_nonzero(dw[-2:])) == 0
    assert int(sum(torch.count_nonzero(part) for part in dw.split(1 << 12))) == 0


def test_capture_of_a_handle_on_the_default_stream_is_refused():
    """Before anything is queued: the capture goes on, and so does the handle."""
    import qml_gradients_amd as hq
    x, w = torch.randn(8, 16, device="cuda"), torch.randn(12, 16, device="cuda")
    layer = hq.Dense(16, 12, 8, stream=0)
    want = layer.forward(x, w)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        twice = x * 2.0
        with pytest.raises(RuntimeError, match="default stream"):
            layer.forward(x, w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(twice, x * 2.0) and torch.equal(layer.forward(x, w), want)


def test_capture_of_a_handle_on_another_stream():
    """Its stream joins the capture; replays, with eager work between, match eager calls."""
    import qml_gradients_amd as hq
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    M, K, N = 130, 300, 70
    layer = hq.Dense(K, N, M, activation="gelu", stream=own.cuda_stream)
    x, w, dy = (torch.randn(*s, device="cuda") for s in ((M, K), (N, K), (M, N)))
    layer.forward(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, z = layer.forward_train(x, w)
        held = (y, *layer.backward(dy, x, w, z))
    for seed in (1, 2, 3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        y, z = layer.forward_train(x, w)
        assert all(torch.equal(a, b) for a, b in zip(got, (y, *layer.backward(dy, x, w, z))))
        torch.cuda.synchronize()


def test_workspace_takes_what_torch_keeps_unused(monkeypatch):
    """Memory that torch's allocator holds and nobody uses is given back before a layer is refused for want of it."""
    import qml_gradients_amd as hq
    create, freed, fail = hq.hqml_dense_create, [], [1]

    def short(cfg):
        if fail[0]:
            fail[0] -= 1
            raise hq.HqmlError(hq.HQML_ERR_OOM, "workspace")
        return create(cfg)

    monkeypatch.setattr(hq, "hqml_dense_create", short)
    empty = torch.cuda.empty_cache
    monkeypatch.setattr(torch.cuda, "empty_cache", lambda: (freed.append(1), empty()))
    layer = hq.Dense(16, 12, 8)
    assert freed and layer.forward(torch.ones(8, 16, device="cuda"), torch.ones(12, 16, device="cuda"))[0, 0] == 16
    fail[0] = 2     # still none: refused
    with pytest.raises(hq.HqmlError) as e:
        hq.Dense(16, 12, 8)
    assert e.value.status == hq.HQML_ERR_OOM and not fail[0]
    with pytest.raises(hq.HqmlError):   # other errors are not tried again
        freed.clear()
        hq.Dense(0, 12, 8)
    assert not freed
