"""Checks on the gfx950 assembly of the W8A8 kernels that no numeric test sees (the
checks of spills and M0 cover every source already).

* Weight stream: a wave waits before the first barrier until its activation loads
  have landed, and for none of the weight loads issued after them.  Fewer loads
  after the last activation load than the wait's count would let the barrier pass
  too early.
* Tiles: the waits of the K loop leave the loads of later steps in flight, and the
  loads sit between the MFMAs of a half step.
* K splits of the stream and of tiles: the hand-off through the workspace uses device-scope
  stores and loads, acknowledged before the counter is raised."""
import re

import pytest

from tests.test_build_registers import _asm, _hipcc, _kernels, _vmcnt

pytestmark = pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")


def _named(pattern):
    for name, ins in _kernels(_asm("gemm_w8a8.hip")):
        m = re.search(pattern, name)
        if m:
            yield name, ins, m


def test_stream_waits_only_for_the_activation_loads():
    seen = 0
    for name, ins, m in _named(r"k_w8a8_streamILi(\d+)ELi(\d+)ELi(\d+)ELb([01])ELb([01])E"):
        allowed = int(m.group(2)) * int(m.group(3))
        last = max(i for i, s in enumerate(ins) if s.startswith("global_load_lds"))
        bar = next(i for i in range(last, len(ins)) if ins[i].startswith("s_barrier"))
        seg = ins[last + 1:bar]
        assert sum(s.startswith("global_load") for s in seg) == allowed, name
        waits = [w for w in map(_vmcnt, (s for s in seg if s.startswith("s_waitcnt"))) if w is not None]
        assert waits and waits[-1] == allowed, f"{name}: waits {waits}, want {allowed}"
        if m.group(4) == "0" or m.group(5) == "1":   # (the dense loops wait before their weight loads too)
            assert min(waits) == allowed, f"{name}: waits {waits}, want {allowed}"
        seen += 1
    assert seen >= 12, seen


def test_tile_loop_keeps_loads_in_flight():
    seen = 0
    for name, ins, m in _named(r"k_w8a8_tileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb([01])ELb([01])E"):
        bm, bn, wm, wn, kg, stages, sub = (int(x) for x in m.groups()[:7])
        dma = sub * (bm + bn) * 64 // (wm * wn * 1024)
        first = next(i for i, s in enumerate(ins) if s.startswith("v_mfma"))
        last = max(i for i, s in enumerate(ins) if s.startswith("v_mfma"))
        waits = [w for w in map(_vmcnt, (s for s in ins[first:last] if s.startswith("s_waitcnt"))) if w is not None]
        assert waits and set(waits) == {(stages - 2) * dma}, f"{name}: waits {sorted(set(waits))}, want {(stages - 2) * dma}"
        run = longest = 0
        for s in ins[first:last + 1]:
            if s.startswith("v_mfma"):
                run += 1
                longest = max(longest, run)
            elif s.startswith(("global_load_lds", "ds_read", "s_barrier")):
                run = 0
        half = (bm // wm // 32) * (bn // wn // 32)
        assert longest <= half, f"{name}: {longest} MFMAs with no load or read between them"
        seen += 1
    assert seen >= 20, seen


def test_split_handoff():
    seen = 0
    for name, ins, _ in _named(r"k_w8a8_streamILi\d+ELi\d+ELi\d+ELb[01]ELb0E|k_w8a8_tileI(Li\d+E)+Lb0ELb[01]ELb1E"):
        a = next(i for i, s in enumerate(ins) if s.startswith("global_atomic_add"))
        dev = [i for i, s in enumerate(ins[:a]) if s.startswith("global_store") and re.search(r"\bsc1\b", s)]
        assert dev, name
        assert any("vmcnt(0)" in s for s in ins[dev[-1] + 1:a] if s.startswith("s_waitcnt")), name
        assert "sc0" in ins[a], name
        assert any(s.startswith("global_load") and re.search(r"\bsc1\b", s) for s in ins[a + 1:]), name
        assert not any(s.startswith(("buffer_wbl2", "buffer_inv")) for s in ins), name
        seen += 1
    assert seen >= 18, seen
