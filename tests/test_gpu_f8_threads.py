"""Several host threads on one stream: every call's result is that of the same call alone."""
import threading

import numpy as np
import pytest

import f8_reference as R

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("side", [False, True])
def test_threads_on_one_stream(cuda_lib, side):
    import torch
    q = cuda_lib
    rng = np.random.default_rng(12)
    E, H, I = 6, 256, 144
    stacks = [[R.weights(rng, n, k) for _ in range(E)] for n, k in ((I, H), (I, H), (H, I))]
    mlp = [_t(np.stack([p[i] for p in s])) for s in stacks for i in (0, 1)]
    W, S = (_t(a) for a in R.weights(rng, 700, 1024))
    st = torch.cuda.Stream() if side else torch.cuda.default_stream()

    def job(seed):
        """Calls of every kind whose launches share the workspace, on data of this thread's own."""
        g = np.random.default_rng(seed)
        few, many = (_t(g.standard_normal((m, 1024)).astype(np.float32)).bfloat16() for m in (40 + seed, 270 + seed))
        logits = _t(g.standard_normal((300 + seed, E)).astype(np.float32))
        x = _t(g.standard_normal((300 + seed, H)).astype(np.float32)).half()

        def run():
            with torch.cuda.stream(st):
                r = q.qmm_route(logits, 2)
                return [q.qmm_f8(W, S, few), q.qmm_f8(W, S, many), *r, q.qmm_f8_moe(x, r, *mlp),
                        q.qmm_f8_experts(mlp[0], mlp[1], x, r.offsets, rows=r.rows)]
        return run
    jobs = [job(s) for s in range(4)]
    torch.cuda.synchronize()
    alone = [j() for j in jobs]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            for _ in range(30):
                got = jobs[i]()
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(alone[i], got)):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and not wrong, (errors, len(wrong))
    assert q.qmm_device_status() == 0
