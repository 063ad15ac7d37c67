"""The layer oracle against the formats and against hand-worked values (CPU)."""
import numpy as np

import oracle
from oracle import layer as ol


def test_value_tables_agree_with_the_gemv_oracle():
    assert np.array_equal(ol.e2m1_values(np.arange(256, dtype=np.uint8))[0::2], oracle.e2m1_table()[np.arange(256) % 16])
    assert np.array_equal(ol.e4m3_values(np.arange(256, dtype=np.uint8)), oracle.e4m3_table(), equal_nan=True)


def test_round_e4m3_is_the_nearest_code():
    codes = np.arange(0x7F, dtype=np.uint8)
    v = ol.e4m3_values(codes)
    assert np.array_equal(ol.round_e4m3(v), codes)
    mid = (v[1:] + v[:-1]) / 2  # ties go to the even code
    want = np.where(codes[1:] % 2 == 0, codes[1:], codes[:-1])
    assert np.array_equal(ol.round_e4m3(mid), want)
    assert np.array_equal(ol.round_e4m3(np.nextafter(mid, 1e9)), codes[1:])
    assert np.array_equal(ol.round_e4m3(np.nextafter(mid, 0)), codes[:-1])
    assert ol.round_e4m3(np.array([1e6]))[0] == 0x7E


def test_round_e2m1_is_the_nearest_code():
    v = ol.E2M1
    mid = (v[1:] + v[:-1]) / 2
    codes = np.arange(8)
    assert np.array_equal(ol.round_e2m1(v), codes)
    assert np.array_equal(ol.round_e2m1(mid), np.where(codes[1:] % 2 == 0, codes[1:], codes[:-1]))
    assert np.array_equal(ol.round_e2m1(np.nextafter(mid, 9)), codes[1:])
    assert ol.round_e2m1(np.array([1e9]))[0] == 7


def test_quantize_by_hand():
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :4] = [6, -6, 1, 0.25]   # s = 1: codes 7, 15, 2, 0 (0.25 ties to 0)
    x[0, 16:18] = [np.inf, 1]
    q, sf = ol.quantize(x)
    assert sf.tolist() == [[0x38, 0x7F]]
    assert q[0, :2].tolist() == [0xF7, 0x02] and not q[0, 2:].any()


def test_atoms_round_trip_and_match_the_repack():
    rng = np.random.default_rng(0)
    for L, rows, kb in ((1, 1, 4), (2, 130, 5), (3, 300, 13)):
        sf = rng.integers(0, 256, (L, rows, kb), dtype=np.uint8)
        flat = ol.atoms(sf)
        assert np.array_equal(flat, oracle.repack_scales(sf, rows, 16 * kb, L))
        assert np.array_equal(ol.from_atoms(flat, rows, kb, L), sf)


def test_route_by_hand():
    x = np.array([[0.0, 2.0, 2.0, 1.0], [-np.inf, np.nan, -np.inf, 3.0], [-np.inf] * 4])
    ids, w, _ = ol.route(x, 2)
    assert ids.tolist() == [[1, 2], [3, -1], [-1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0]])
    # groups {0,1} and {2,3}: 0.9 + 0.1 against 0.6 + 0.5 (sigmoid of the logits)
    x = np.log(np.array([[9.0, 1 / 9, 1.5, 1.0]]))
    assert ol.route(x, 2, sigmoid=True, groups=2, top_groups=1)[0].tolist() == [[2, 3]]
    assert ol.route(x, 1, sigmoid=True, bias=np.array([0.0, 0.0, 0.0, 0.5]))[0].tolist() == [[3]]


def test_moe_rows_by_hand():
    ids = np.array([[2, 0], [2, -1], [2, 5], [0, 2]])
    rows, counts, starts = ol.moe_rows(ids, 3, 2)
    assert counts.tolist() == [2, 0, 4] and starts.tolist() == [0, 128, 128]
    assert rows.tolist() == [[128, 0], [129, -1], [256, -1], [1, 257]]
