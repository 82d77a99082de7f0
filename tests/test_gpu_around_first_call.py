"""Calls around the layer made for the first time in a process while a graph is captured, and from several
host threads at once."""

import os
import subprocess
import sys
import threading

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from test_gpu_balance import make as balance_make
from test_gpu_gemv import make as gemv_make
from test_gpu_norm import make as norm_make

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.path.insert(0, "tests")
import torch
from test_gpu_around_first_call import Calls
calls = Calls()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    calls.run()
graph.replay()
torch.cuda.synchronize()
got = [v.clone() for v in calls.outputs()]
calls.clear()
calls.run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls.outputs()))
print("same")
"""


class Calls:
    """One call of each operator: large enough for the forms that ask for more shared memory."""

    def __init__(self, seed=0):
        self.norm, t, _ = norm_make(700, 2048, y="bf16", post=True, kind="channel", seed=seed)
        self.t = t
        self.n = {k: torch.empty_like(t[k]) for k in ("h", "dh_out", "y")}
        self.x = torch.empty_like(t["dx"])
        self.w = [torch.empty(2048, device="cuda") for _ in range(3)]
        self.ws = smg.new_norm_workspace(self.norm, 700)
        self.logits, self.ids, _ = balance_make(3000, 512, 10, "bf16", seed=seed)
        self.loss, self.prob = torch.empty(2, device="cuda"), torch.empty(512, device="cuda")
        self.counts = torch.empty(512, device="cuda", dtype=torch.int32)
        self.rows = torch.empty(1, device="cuda", dtype=torch.int32)
        self.grad, self.dl = torch.ones(2, device="cuda"), torch.empty_like(self.logits)
        self.bws = smg.new_balance_workspace(3000, 512)
        self.mats = [(smg.Matrix(w, s, w.shape[0], x.shape[1]), x, torch.empty(x.shape[0], w.shape[0], device="cuda"))
                     for w, s, x in (gemv_make(5000, 1024, T, seed=seed) for T in (1, 4, 13))]

    def run(self):
        t, n = self.t, self.n
        smg.redmoe_norm_forward(self.norm, t["h"], h_out=n["h"], x=self.x, y=t["y"], gate=t["gate"])
        smg.redmoe_norm_backward(self.norm, t["h"], n["dh_out"], self.ws, dh_out=t["dh_out"], dx=t["dx"], y=t["y"],
                                 gate=t["gate"], dy=n["y"], dgate=self.w[0], dpost_w=self.w[1], dpre_w=self.w[2])
        smg.redmoe_balance_forward(self.logits, self.ids, self.loss, self.counts, self.prob, self.rows, self.bws)
        smg.redmoe_balance_backward(self.logits, self.counts, self.rows, self.grad, self.dl, 10)
        for m, x, y in self.mats:
            smg.redmoe_gemv(m, x, y)

    def outputs(self):
        return [*self.n.values(), self.x, *self.w, self.loss, self.prob, self.counts, self.rows, self.dl,
                *(y for _, _, y in self.mats)]

    def clear(self):
        for v in self.outputs():
            v.fill_(-1)


def test_first_calls_of_a_process_inside_a_capture(gpu_lib):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-3000:]


def test_calls_from_several_threads(gpu_lib):
    calls = [Calls(seed=i) for i in range(4)]
    want = []
    for c in calls:
        c.run()
        torch.cuda.synchronize()
        want.append([v.clone() for v in c.outputs()])
        c.clear()
    torch.cuda.synchronize()
    streams, errors = [torch.cuda.Stream() for _ in calls], []

    def work(c, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(30):
                    c.run()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c.outputs(), w))
