"""Workspaces that pass from op to op: what one op leaves there is never taken
for a look-back record of a later one, whatever its values."""
from __future__ import annotations

import pytest
import torch

from linear_recurrence_scans_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"
CONTROL = 256


def _epoch(ws, value=None):
    words = ws[8:16].view(torch.int64)
    if value is not None:
        words.fill_(value)
    return int(words)


def _scans(mg, ws_bytes):
    """Calls that read tagged records, by name: f(ws) -> outputs."""
    a, b, gA, gB = (t.to(DEV) for t in wl.mingru_linear(2, 4096, 256, seed=41))
    A, Bc = mg.linear_scan_fwd(a, b)
    lc, lv = (t.to(DEV) for t in wl.mingru_log(2, 4096, 256, seed=42))
    x1, x2 = (t.to(DEV) for t in wl.mingru_x(2, 4096, 256, seed=43)[:2])
    cu = torch.tensor([0, 7, 2100, 4096], device=DEV)
    assert ws_bytes >= max(mg.linear_workspace_size(2, 4096, 256), mg.log_workspace_size(2, 4096, 256),
                           mg.mingru_workspace_size(2, 4096, 256), mg.varlen_workspace_size(4096, 256))
    oa, ob, og = (t[..., :255].contiguous() for t in (a, b, gB))   # one channel a lane
    oA, oBc = mg.linear_scan_fwd(oa, ob)
    return {
        "linear": lambda ws: mg.linear_scan_fwd(a, b, ws=ws),
        "linear odd": lambda ws: mg.linear_scan_fwd(oa, ob, ws=ws),
        "linear odd bwd": lambda ws: mg.linear_scan_bwd(oa, oA, oBc, og, og, ws=ws),
        "linear bf16": lambda ws: mg.linear_scan_fwd(a.bfloat16(), b.bfloat16(), ws=ws),
        "linear bwd": lambda ws: mg.linear_scan_bwd(a, A, Bc, gA, gB, ws=ws),
        "log": lambda ws: (mg.parallel_scan_log_fwd(lc, lv, ws=ws),),
        "mingru": lambda ws: mg.mingru_scan_fwd(x1, x2, ws=ws),
        "varlen": lambda ws: mg.linear_scan_varlen_fwd(a[0], b[0], cu, ws=ws),
    }


def test_partial_sums_of_two_are_no_record(cuda_lib):
    """Gradients of a norm whose upstream gradient is 1: every partial sum of its
    bias gradient is 2.0 where a block has two rows.  The first scan on that
    workspace does not take them for its predecessors' prefixes."""
    mg = cuda_lib
    x, z = (torch.randn(608, 4096, device=DEV).bfloat16() for _ in range(2))
    w = torch.ones(4096, device=DEV)
    _, stats = mg.group_norm_fwd(x, w, None, z, rms=True, gate_first=True)
    size = 64 << 20
    own = mg.new_workspace(size, DEV)
    for name, scan in _scans(mg, size).items():
        want = scan(own)
        for _ in range(4):
            ws = mg.new_workspace(size, DEV)
            mg.group_norm_bwd(torch.ones_like(x), stats, x, w, None, z, rms=True, gate_first=True, ws=ws)
            got = scan(ws)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), name
            mg.workspace_status(ws)


@pytest.mark.parametrize("value", [2.0, 2.0 + 2.0 ** -22, 0.0, -0.0, float("inf"), float("nan"), -float("inf")])
def test_no_value_is_a_record(cuda_lib, value):
    """The whole workspace behind its control block holds one float."""
    mg = cuda_lib
    size = 64 << 20
    own = mg.new_workspace(size, DEV)
    for name, scan in _scans(mg, size).items():
        want = scan(own)
        ws = mg.new_workspace(size, DEV)
        for _ in range(2):
            ws[CONTROL:].view(torch.float32).fill_(value)
            got = scan(ws)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (name, value)
            mg.workspace_status(ws)


def _tagged_words(mg, ws, epoch, value):
    """Fills the workspace behind its control block with `value` in words tagged
    as those of launch `epoch`."""
    bits = torch.tensor(value).view(torch.int32).item()
    words = ws[CONTROL:].view(torch.int64).view(-1, 2)
    for odd in (0, 1):
        words[:, odd] = (mg.load().mg_testing_record_tag(epoch, odd) - (1 << 32) << 32) | bits


@pytest.mark.parametrize("epoch", [(1 << 21) - 1, 1 << 21, 3 << 21, (1 << 42) - 2])
def test_records_of_earlier_launches_are_not_taken(cuda_lib, epoch):
    """Words of launches whose numbers agree with the running one's in the even
    or in the odd places' bits; across the numbers at which these begin again."""
    mg = cuda_lib
    size = 64 << 20
    own = mg.new_workspace(size, DEV)
    for name, scan in _scans(mg, size).items():
        want = scan(own)
        for older in (epoch - (1 << 21), epoch - 1, epoch ^ 1, epoch ^ (1 << 41)):
            ws = mg.new_workspace(size, DEV)
            _epoch(ws, epoch)
            for k in range(2):
                _tagged_words(mg, ws, (older + k) % (1 << 64), 7.0)
                got = scan(ws)
                assert all(torch.equal(p, q) for p, q in zip(got, want)), (name, older)
            assert _epoch(ws) == epoch + 2
            mg.workspace_status(ws)


def test_a_replayed_graph_writes_no_memory_of_others(cuda_lib):
    """A graph captured on a stream's cached workspace, replayed after a larger
    call replaced that workspace and other tensors took free memory."""
    mg = cuda_lib
    x, dt = torch.randn(2, 200, 96, device=DEV), torch.randn(2, 200, 96, device=DEV)
    A, bc = -torch.rand(96, 16, device=DEV) - 0.1, torch.randn(2, 200, 16, device=DEV)
    side = torch.cuda.Stream()
    key = (0, side.cuda_stream)

    def step():
        y, _, saved = mg.selective_scan_fwd(x, dt, A, bc, bc, save=True)
        return (y, *mg.selective_scan_bwd(y, saved, x, dt, A, bc, bc)[:5])

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    size = mg._ws_cache[key].numel()
    with torch.cuda.stream(side):
        big = torch.randn(4, 2048, 512, device=DEV)
        mg.causal_conv_bwd(big, big, torch.randn(512, 8, device=DEV))
        bb = torch.randn(4, 2048, 16, device=DEV)
        y, _, saved = mg.selective_scan_fwd(big, big, -torch.rand(512, 16, device=DEV), bb, bb, save=True)
        mg.selective_scan_bwd(y, saved, big, big, -torch.rand(512, 16, device=DEV), bb, bb)
        assert mg._ws_cache[key].numel() > size
        del y, saved, big, bb
        others = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (size, size // 2, size, 4 * size) * 4]
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in others)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    mg.workspace_status()
