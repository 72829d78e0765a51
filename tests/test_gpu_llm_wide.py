"""The norm's gradient on wide rows, whose weight-gradient sums lie in shared memory: the first call of a process at
every size (an earlier, wider one can leave a kernel more shared memory than it asked for), and calls from two threads.

Tolerances as in test_gpu_llm_norm: (ranks + 160) 2^-24 of the terms' magnitudes and the output's rounding for dx,
(rows + ranks + 16) 2^-24 of them for dweight."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from collective_fusedallreduce_gb300 import coco

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
E = 2.0 ** -24


def gradient(n, rows, cols, dtype, seed=711):
    """Arguments of a call, and its check."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    dn, dh, hid, w = [rnd(rows, cols) for _ in range(n)], rnd(rows, cols), rnd(rows, cols), rnd(cols)
    rstd = (hid.double().square().mean(-1) + 1e-5).rsqrt().float()
    dx, dw = torch.empty_like(hid), torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    args = (coco.local(dn), coco.replicated([dh] * n), coco.replicated([hid] * n), w, rstd, coco.replicated([dx] * n),
            dw, ws)

    def check():
        r, d = rstd.double()[:, None], sum(x.double() for x in dn)
        xhat, gw = hid.double() * r, d * w.double()
        want = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) + dh.double()
        mag = sum(x.double().abs() for x in dn)
        gm = mag * w.double().abs()
        terms = r * (gm + xhat.abs() * (gm * xhat.abs()).mean(-1, keepdim=True)) + dh.double().abs()
        bound = want.abs() * (torch.finfo(dtype).eps / 2 * 1.01) + (n + 160) * E * terms + 2.0 ** -25
        assert bool(((dx.double() - want).abs() <= bound).all()), ("dx", n, rows, cols, dtype)
        bound = (rows + n + 16) * E * (mag * xhat.abs()).sum(0)
        assert bool(((dw.double() - (d * xhat).sum(0)).abs() <= bound).all()), ("dweight", n, rows, cols, dtype)

    return args, check


def first_calls(cols):
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        for n in (1, 2, 8):
            args, check = gradient(n, 3, cols, dtype)
            coco.coco_allreduce_rmsnorm_backward(*args)
            coco.coco_device_status()
            check()


@pytest.mark.parametrize("cols", [8200, 12224, 12240, 12288, 12296, 16384, 16392, 32768])
def test_first_call_of_a_process(cols):
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"import sys; sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]; " \
           f"import test_gpu_llm_wide as t; t.first_calls({cols})"
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_of_two_threads_do_not_take_each_others_shared_memory(dtype):
    failed = []

    def work(cols):
        try:
            torch.cuda.set_device(DEV)
            s = torch.cuda.Stream()
            args, check = calls[cols]
            for _ in range(2000):
                coco.coco_allreduce_rmsnorm_backward(*args, stream=s)
            s.synchronize()
            check()
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            failed.append((cols, e))

    calls = {cols: gradient(2, 1, cols, dtype) for cols in (32768, 16400)}
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(cols,)) for cols in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [8192, 16384, 16400, 32768])
@pytest.mark.parametrize("place", ["dhidden", "hidden", "dnormed"])
def test_in_place_on_rows_that_are_read_again(dtype, cols, place):
    """Wide rows read dhidden late and the widest hidden twice: dx may still take their place."""
    n, rows = 2, 5
    args, check = gradient(n, rows, cols, dtype)
    coco.coco_allreduce_rmsnorm_backward(*args)
    torch.cuda.synchronize()
    check()
    dn, dh, hid, w, rstd, dx, dw, ws = args
    want, want_dw = dx.tensors[0].clone(), dw.clone()
    to = {"dhidden": dh, "hidden": hid, "dnormed": coco.replicated([dn.tensors[1]] * n)}[place]
    coco.coco_allreduce_rmsnorm_backward(dn, dh, hid, w, rstd, to, dw, ws)
    coco.coco_device_status()
    assert torch.equal(to.tensors[0], want) and torch.equal(dw, want_dw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("groups,n,rows,cols", [(3, 2, 7, 144), (2, 3, 200, 1040), (2, 2, 4, 16400), (32, 2, 40, 64)])
def test_groups_join_in_the_weights_gradient(dtype, groups, n, rows, cols):
    g = torch.Generator(device=DEV).manual_seed(712)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    dn = [rnd(rows, cols) for _ in range(groups * n)]
    hid, w = [rnd(rows, cols) for _ in range(groups)], rnd(cols)
    rstd = torch.stack([(h.double().square().mean(-1) + 1e-5).rsqrt() for h in hid]).float()
    dx, dw = [torch.empty_like(h) for h in hid], torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(groups * rows, cols), dtype=torch.uint8, device=DEV)
    rep = lambda ts: coco.replicated([t for t in ts for _ in range(n)], groups)  # noqa: E731
    coco.coco_allreduce_rmsnorm_backward(coco.local(dn, groups), None, rep(hid), w, rstd, rep(dx), dw, ws)
    coco.coco_device_status()
    want_w, mag_w = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    for i in range(groups):
        mine = dn[i * n:(i + 1) * n]
        r, d, mag = rstd[i].double()[:, None], sum(x.double() for x in mine), sum(x.double().abs() for x in mine)
        xhat, gw, gm = hid[i].double() * r, d * w.double(), mag * w.double().abs()
        want = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
        terms = r * (gm + xhat.abs() * (gm * xhat.abs()).mean(-1, keepdim=True))
        bound = want.abs() * (torch.finfo(dtype).eps / 2 * 1.01) + (n + 160) * E * terms + 2.0 ** -25
        assert bool(((dx[i].double() - want).abs() <= bound).all()), i
        want_w += (d * xhat).sum(0)
        mag_w += (mag * xhat.abs()).sum(0)
    assert bool(((dw.double() - want_w).abs() <= (groups * rows + n + 16) * E * mag_w).all())
