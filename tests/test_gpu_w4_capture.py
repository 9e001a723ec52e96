"""The 4-bit and logit calls whose first call of all is captured into a graph, in a process of its own; and two captured graphs that
run at the same time."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path.insert(0, {root!r})
import torch
import verify_head_gb300 as vh
vh.build()
g = torch.Generator('cuda').manual_seed(0)
dev, u8 = 'cuda', torch.uint8


class Step:
    # T = 1024 rows of 8192 columns take the CTA pairs, 4 of 500 a cluster for each tile, 4 of 30000 and 100 one CTA
    def __init__(self, T, V, H):
        self.size = T, V, H
        self.x = torch.randn(T, H, generator=g, device=dev).bfloat16()
        self.w = torch.randn(V, H, generator=g, device=dev).bfloat16()
        self.codes, self.scales = torch.empty(V, H // 2, dtype=u8, device=dev), torch.empty(V, H // 16, dtype=u8, device=dev)
        self.wt, self.xt = (torch.empty(vh.vh_nvfp4_tiles_bytes(n, H), dtype=u8, device=dev) for n in (V, T))
        self.rs, self.y = torch.empty(T, device=dev), torch.empty(T, V, device=dev)
        self.back = torch.empty(V, H, device=dev).bfloat16()
        S = max(1, T // 4)
        one = torch.ones(S, device=dev)
        self.rules = dict(history=torch.randint(0, V, (S, 300), generator=g, device=dev, dtype=torch.int32), repetition=one * 1.2,
                          frequency=one * 0.3, temperature=one * 0.7)
        self.out, self.d = torch.empty_like(self.y), torch.empty_like(self.y)

    def run(self):
        T, V, H = self.size
        vh.nvfp4_quantize(self.w, 0.002, self.codes, self.scales)
        vh.nvfp4_tile(self.codes, self.scales, tiles=self.wt)
        vh.nvfp4_dequantize(self.codes, self.scales, 0.002, out=self.back)
        vh.nvfp4_quantize_tiles(self.x, tiles=self.xt, row_scales=self.rs)
        vh.nvfp4_matmul(self.xt, self.rs, self.wt, 0.002, T, V, H, out=self.y)
        vh.logits_process(self.y, out=self.out, **self.rules)
        vh.logits_process_grad(self.y, self.out, dlogits=self.d, **self.rules)

    def results(self):
        return [t.clone() for t in (self.codes, self.wt, self.back, self.y, self.out, self.d)]


steps = [Step(4, 500, 4096), Step(4, 30000, 512), Step(100, 3000, 256), Step(1024, 8192, 2048)]
torch.cuda.synchronize()
graphs = []
for s in steps:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    graphs.append(graph)
for graph in graphs:
    graph.replay()
torch.cuda.synchronize()
captured = [s.results() for s in steps]
streams = [torch.cuda.Stream() for _ in steps]
for i in range(10):
    for s in steps:
        for t in (s.codes, s.wt, s.xt, s.back, s.y, s.out, s.d):
            t.zero_()
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for s, want in zip(steps, captured):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want)), s.size
for s, want in zip(steps, captured):
    for t in (s.codes, s.wt, s.back, s.y, s.out, s.d):
        t.zero_()
    s.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.results(), want)), s.size
    assert float(s.y.abs().max()) > 0 and float(s.d.abs().max()) > 0
print('captured')
"""


def test_first_call_in_a_graph_and_graphs_side_by_side():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CODE.format(root=ROOT)], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    assert "captured" in r.stdout
