"""Host threads that call a kernel at once, each on its own stream, whose
shared memory differs with the sizes of the call: what one thread's launch
allows must not fall below another's."""

import threading

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu


def test_few_tokens_of_different_sizes_at_once(W):
    from w8a16_linear_gb300 import binding as b
    shapes = [(1, 256, 128), (128, 256, 128), (16, 256, 20480), (128, 512, 512)]   # 144, 198, 113 and 198 KB
    cases = []
    for M, K, N in shapes:
        g = torch.Generator(device="cuda").manual_seed(M + N)
        x, w = ((torch.randn(s, generator=g, device="cuda") * 50).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for s in ((M, K), (N, K)))
        st, sc = torch.rand((M,), generator=g, device="cuda"), torch.rand((N,), generator=g, device="cuda")
        want = W.fp8_linear_w8a8_pertoken(x, st, w, sc)
        cases.append((x, st, w, sc, want))
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(cases))

    def work(i):
        x, st, w, sc, want = cases[i]
        stream, y = torch.cuda.Stream(), torch.zeros_like(want)
        # the C entry itself: no interpreter between two launches but the loop
        M, K, N = shapes[i]
        ptr, num = b.ctypes.c_void_p * 1, b.ctypes.c_int64 * 1
        args = (x.data_ptr(), M, K, st.data_ptr(), 1, ptr(w.data_ptr()), num(N), ptr(sc.data_ptr()), ptr(y.data_ptr()),
                stream.cuda_stream)
        call = b.lib().fp8_linear_w8a8_pertoken
        torch.cuda.synchronize()
        start.wait()
        for k in range(4000):
            status = call(*args)
            if status != 0:
                failures.append((shapes[i], k, status, b.lib().w8_last_error()))
                break
        stream.synchronize()
        if not torch.equal(y.view(torch.int16), want.view(torch.int16)):
            failures.append((shapes[i], "bits"))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    W.poll_device_error()
    assert not failures, failures


def test_modulated_norms_of_different_widths_at_once(W):
    from w8a16_linear_gb300 import binding as b
    widths = [520, 1016, 2056, 4088]      # two to a kernel
    cases = []
    for K in widths:
        g = torch.Generator(device="cuda").manual_seed(K)
        x, shift, scale = (torch.randn((n, K), generator=g, device="cuda").bfloat16() for n in (64, 2, 2))
        s_in = torch.full((1,), 0.01, device="cuda")
        cases.append((x, shift, scale, s_in, W.ln_modulate_quant(x, shift, scale, s_in)))
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(cases))

    def work(i):
        x, shift, scale, s_in, want = cases[i]
        stream, q = torch.cuda.Stream(), torch.zeros_like(want)
        torch.cuda.synchronize()
        args = (x.data_ptr(), 64, widths[i], shift.data_ptr(), scale.data_ptr(), 32, 1e-6, s_in.data_ptr(), q.data_ptr(), None,
                stream.cuda_stream)
        call = b.lib().ln_modulate_quant
        start.wait()
        for k in range(4000):
            status = call(*args)
            if status != 0:
                failures.append((widths[i], k, status, b.lib().w8_last_error()))
                break
        stream.synchronize()
        if not torch.equal(q, want):
            failures.append((widths[i], "bits"))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    W.poll_device_error()
    assert not failures, failures
