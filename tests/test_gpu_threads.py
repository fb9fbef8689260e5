"""Two host threads that call at the same time, each on its own stream and with
its own workspace and output.  ctypes releases the interpreter's lock in a call,
so their launches interleave; neither may change what the other's launch is
allowed to take, nor its result."""
import threading

import pytest
import torch

import w8a8_activation_quantized_b200 as cider
from tests.paged_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _at_once(calls, times):
    """Runs each of `calls` `times` times in a thread of its own, all started
    together; the first exception of any of them is raised."""
    start, errors = threading.Barrier(len(calls)), []

    def work(call):
        start.wait()
        try:
            for _ in range(times):
                call()
                if errors:
                    return
        except Exception as e:  # noqa: BLE001 (raised below, in the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("what", ["paged 16-row tiles", "paged tensor-core tiles", "decode attention", "per-channel product"])
def test_a_thread_whose_first_use_of_cuda_is_the_call(what):
    """Everything is allocated beforehand, so the thread makes no other call first."""
    g = torch.Generator(device="cuda").manual_seed(5)
    stream = torch.cuda.Stream()
    if what.startswith("paged"):
        cider.cider_test_set_paged_kernel(1 if "16" in what else 2)
        b = Batch([(300, 40), (40, 1)], 8, 2, D=64, page=32, seed=3)
        ws = torch.empty(cider.cider_paged_attention_workspace_bytes(b.T, 2, 8, 2, 64, 40), dtype=torch.uint8, device="cuda")

        def call(out, st):
            return b.run(cider, out=out, workspace=ws, stream=st)
        like = b.q
    elif what == "decode attention":
        q, k, v = (torch.randn(s, generator=g, device="cuda").half() for s in ((8, 128), (2, 500, 128), (2, 500, 128)))
        ws = torch.empty(cider.cider_sdpa_decode_workspace_bytes(8, 2, 500, 128), dtype=torch.uint8, device="cuda")

        def call(out, st):
            return cider.cider_sdpa_decode(q, k, v, out=out, workspace=ws, stream=st)
        like = q
    else:
        x, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((200, 256), (264, 256)))
        sx, sw = (torch.rand(n, generator=g, device="cuda") for n in (200, 264))

        def call(out, st):
            return cider.cider_w8a8_gemm_pc_q(x, sx, w, sw, y=out, stream=st)
        like = torch.empty((200, 264), dtype=torch.float16, device="cuda")
    try:
        want, out = torch.zeros_like(like), torch.zeros_like(like)
        torch.cuda.synchronize()
        call(want, stream)
        torch.cuda.synchronize()
        _at_once([lambda: call(out, stream)], 1)
        assert torch.equal(out, want)
    finally:
        cider.cider_test_set_paged_kernel(0)


@pytest.mark.parametrize("kernel", [1, 2])
def test_paged_attention_of_small_and_large_batches(kernel, monkeypatch):
    """The kernels' shared memory grows with the number of requests.  The calls
    go to the library as the binding makes them, but back to back, so that they
    meet often."""
    cider.cider_test_set_paged_kernel(kernel)
    try:
        large = [(i % 40, 1) if i % 512 == 511 else (0, 0) for i in range(4096)]
        bs = [Batch(lens, 8, 2, D=64, page=32, seed=i) for i, lens in enumerate(([(40, 1)], large, [(17, 1)], large))]
        want = [b.run(cider) for b in bs]
        outs = [torch.zeros_like(w) for w in want]
        ws = [torch.empty(cider.cider_paged_attention_workspace_bytes(b.T, len(b.lens), 8, 2, 64, 1), dtype=torch.uint8,
                          device="cuda") for b in bs]
        streams = [torch.cuda.Stream() for _ in bs]
        made = []
        monkeypatch.setattr(cider, "_paged_call", lambda name, index, stream, *args: made.append((name, args, stream)))
        for b, o, w, s in zip(bs, outs, ws, streams):
            b.run(cider, out=o, workspace=w, stream=s)
        monkeypatch.undo()
        torch.cuda.synchronize()

        def calls(name, args, stream):
            f, st = getattr(cider.lib(), name), stream.cuda_stream

            def some():
                for _ in range(100):
                    status = f(*args, st)
                    if status != 0:
                        cider._check(name, status)
                stream.synchronize()
            return some
        _at_once([calls(*m) for m in made], 100)
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        cider.cider_device_status()
    finally:
        cider.cider_test_set_paged_kernel(0)


@pytest.mark.parametrize("product", ["w8a8", "w8a16"])
@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
def test_decode_products_of_few_and_more_rows(kernel, product):
    """The decode kernels' shared memory grows with the rows.  Calls back to
    back, straight to the library."""
    cider.cider_test_set_small_m_kernel(kernel)
    try:
        g = torch.Generator(device="cuda").manual_seed(7)
        N, K = 520, 10240
        w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        sw = torch.rand(N, generator=g, device="cuda")
        xs = [torch.randn((M, K), generator=g, device="cuda").half() for M in (2, 4, 2, 4)]
        f = getattr(cider.lib(), "cider_w8a8_linear_pc" if product == "w8a8" else "cider_w8a16_mv_pc")
        call = cider.cider_w8a8_linear_pc if product == "w8a8" else cider.cider_w8a16_mv_pc
        want = [call(x, w, sw) for x in xs]
        ys = [torch.zeros_like(y) for y in want]
        streams = [torch.cuda.Stream() for _ in xs]
        torch.cuda.synchronize()

        def calls(x, y, stream):
            a = [x.data_ptr(), cider._DT[x.dtype], x.shape[0], K, w.data_ptr(), sw.data_ptr(), N, y.data_ptr(),
                 cider._DT[y.dtype]] + ([None, 0] if product == "w8a8" else []) + [stream.cuda_stream]

            def some():
                for _ in range(100):
                    status = f(*a)
                    if status != 0:
                        cider._check(f.__name__, status)
                stream.synchronize()
            return some
        _at_once([calls(*m) for m in zip(xs, ys, streams)], 100)
        assert all(torch.equal(y, v) for y, v in zip(ys, want))
        cider.cider_device_status()
    finally:
        cider.cider_test_set_small_m_kernel(0)
