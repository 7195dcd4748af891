"""Calls from several threads: autograd runs the lane's backward passes on
threads of its own, beside the calls of the program's thread."""
import ctypes
import threading

import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def in_thread(f):
    """f() on a thread of its own; its exception, if any, is raised here."""
    failed = []

    def work():
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if failed:
        raise failed[0]


def test_binding_belongs_to_its_thread():
    """Between a thread's binding and its call another thread binds a stream of
    its own.  The call still goes to the first stream, which is shown by its
    being captured there: nothing runs before the graph does."""
    lib = mo.lib()
    rows, dim = 4, 64
    x = torch.randn(rows, dim, device=DEV)
    want = mo.muon_layer_norm(x)[0]
    y, mean, rstd = torch.full_like(x, 7.0), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    vp = ctypes.c_void_p
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1, capture_error_mode="thread_local"):
        assert lib.muon_set_stream(vp(s1.cuda_stream)) == mo.MUON_OK
        in_thread(lambda: lib.muon_set_stream(vp(s2.cuda_stream)))
        rc = lib.muon_layer_norm(vp(x.data_ptr()), mo.MUON_DTYPE_F32, dim, rows, dim, None, None, mo.MUON_DTYPE_F32,
                                 1e-5, vp(y.data_ptr()), vp(mean.data_ptr()), vp(rstd.data_ptr()))
        assert rc == mo.MUON_OK
    torch.cuda.synchronize()
    assert (y == 7).all()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # a thread that has bound nothing uses the last binding
    y.fill_(7)
    lib.muon_set_stream(vp(s2.cuda_stream))
    torch.cuda.synchronize()
    in_thread(lambda: lib.muon_layer_norm(vp(x.data_ptr()), mo.MUON_DTYPE_F32, dim, rows, dim, None, None,
                                          mo.MUON_DTYPE_F32, 1e-5, vp(y.data_ptr()), vp(mean.data_ptr()),
                                          vp(rstd.data_ptr())))
    s2.synchronize()
    assert torch.equal(y, want)


def test_steps_beside_backward_calls_on_another_thread():
    """One thread steps AdamW on its stream while another runs the lane's
    backward calls on its own: each gets what it gets alone."""
    def adam(n):
        p = [torch.linspace(-1, 1, 5000, device=DEV)]
        g = [torch.linspace(1, -2, 5000, device=DEV)]
        m, v = [torch.zeros(5000, device=DEV)], [torch.zeros(5000, device=DEV)]
        for i in range(n):
            mo.muon_adamw_step(p, g, m, v, i + 1)
        return p[0]

    gen = torch.Generator(device=DEV).manual_seed(1)
    t = torch.randint(0, 700, (3000,), generator=gen, device=DEV)
    g = torch.randn(3000, 64, generator=gen, device=DEV)
    x = torch.randn(3000, 64, generator=gen, device=DEV)
    _, mean, rstd = mo.muon_layer_norm(x)

    def lane():
        dx, _, db = mo.muon_layer_norm_backward(g, x, mean, rstd)
        return dx, db, mo.muon_embedding_backward(t, dx, 700)

    mo.muon_set_config(grad_dtype=mo.MUON_DTYPE_F32, param_dtype=mo.MUON_DTYPE_F32)
    try:
        want_p, want_l = adam(200), lane()
        torch.cuda.synchronize()
        got = {}
        start = threading.Barrier(2)

        def stepper():
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                got["p"] = adam(200)
                torch.cuda.current_stream().synchronize()

        def backward():
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                got["l"] = [lane() for _ in range(200)]
                torch.cuda.current_stream().synchronize()

        threads = [threading.Thread(target=f) for f in (stepper, backward)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        assert torch.equal(got["p"], want_p)
        for out in got["l"]:
            for a, b in zip(out, want_l):
                assert torch.equal(a, b)
    finally:
        mo.muon_reset_config()
    assert mo.muon_device_status(DEV) == (mo.MUON_OK, -1)
