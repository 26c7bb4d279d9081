"""CPU tests of a ChunkLayout as it is made."""
import position_independent_kv_critical_gb300 as pcf


def test_no_row_has_a_slot_before_the_first_tables():
    L = pcf.ChunkLayout(3, 8, 2, 64, 40, 512, max_pages=8, max_rows=20, max_chunk=9, device="cpu")
    assert L.slot_map.tolist() == [-1] * 20 and L.row_pos.tolist() == [-1] * 20
    assert not L.row_base.any() and not L.plan.any()
