"""The 8-bit linear layers' calls by several threads at once: every thread's every
result is compared, and a thread that fails or hangs fails the test."""
import pytest

pytestmark = pytest.mark.gpu
THREADS, TURNS = 3, 3


@pytest.mark.parametrize("shared", [False, True])
def test_every_result_of_every_thread(shared):
    """On a stream of each thread, and all on one."""
    import threading

    import torch
    from test_linear8_gpu import _bytes, _calls, _same
    calls = _calls(30)
    want = [_bytes(f()) for _, f in calls]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    wrong, compared = [], [0] * THREADS
    start = threading.Barrier(THREADS)

    def work(i):
        try:
            stream = one if shared else torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(TURNS):
                    got = [_bytes(f()) for _, f in calls]
                    stream.synchronize()
                    for (name, _f), g, w in zip(calls, got, want):
                        if not _same(g, w):
                            wrong.append((i, name))
                        compared[i] += 1
        except BaseException as e:
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,), daemon=True) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads), "a thread did not end"
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert compared == [TURNS * len(calls)] * THREADS
