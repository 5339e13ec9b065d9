"""How the sequence operators' launches are cut (CPU only: csrc/sequence_plan.h built with g++ under the sanitizers,
for 256 CUs): the sizes of the GPU tests reach every form of the kernels, plans cover their work, and the
ends of the accepted sizes overflow nothing."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_weight_direct_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-I" + CSRC,
                    "-I" + os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "sanitize", "sequence_plans.cpp"), "-o", exe],
                   check=True)

    def run(*calls):
        r = subprocess.run([exe], input="\n".join(" ".join(str(v) for v in c) for c in calls), capture_output=True, text=True,
                           check=True, timeout=60)
        return [{k: int(v) for k, v in (f.split("=") for f in line.split())} for line in r.stdout.splitlines()]
    return run


def _scan_forms(p):
    """The kernels a scan's prompt runs: (positions a lane, first pass, reading ahead)."""
    return {(p["ti"], False, bool(p["ahead"]))} | ({(p["ti"], True, bool(p["ahead"]))} if p["segments"] > 1 else set())


def test_both_forms_of_the_convolution_are_tested(plans):
    """test_conv_long_rows: 1700, 2041, 2048, 2049 and 4090 positions."""
    lengths = (1700, 2041, 2048, 2049, 4090)
    for dtype, own in ((0, [1, 1, 1, 0, 0]), (1, [0, 1, 1, 0, 1]), (2, [0, 1, 1, 0, 1])):
        p = plans(*(("conv", dtype, 2, 3, L) for L in lengths))
        assert [v["own"] for v in p] == own and [v["places"] for v in p] == [-(-L // 8) for L in lengths]


def test_every_form_of_the_scan_is_tested(plans):
    sizes = [("scan", 2, 5, 64, 16, 1), ("scan", 2, 5, 300, 16, 1), ("scan", 2, 5, 1025, 16, 1), ("scan", 2, 19, 512, 16, 1),
             ("scan", 9, 1023, 520, 20, 1), ("scan", 9, 1023, 520, 16, 1), ("scan", 2, 512, 2311, 20, 1), ("scan", 1, 1024, 2500, 16, 4)]
    p = plans(*sizes)
    assert set().union(*map(_scan_forms, p)) == {(4, False, False), (8, False, False), (16, False, False), (16, True, False),
                                                 (16, False, True), (16, True, True)}
    for k in (4, 5):  # tests of the form without reading ahead, in one walk
        assert _scan_forms(p[k]) == {(16, False, False)}
    for k in (6, 7):  # and in segments
        assert _scan_forms(p[k]) == {(16, False, False), (16, True, False)} and p[k]["segments"] > 2


def test_every_form_of_the_second_product_is_tested(plans):
    """test_adapter_tiles_side_by_side: four tiles side by side, the last set of them cut short, in every type;
    test_adapter_pieces_of_the_channels: 4 and 2 pieces of C; the other adapter tests: one tile, 1 and 4 pieces."""
    for dtype, tile in ((0, 64), (1, 128), (2, 128)):
        for R in (4, 16):
            p = plans(("adapter", dtype, 64, 12, 150, 21 * tile - 37, R))[0]
            assert p["wide"] and p["ltiles"] == 21 and p["mtiles"] == 2 and p["segments"] == 1
        p = plans(("adapter", dtype, 8, 1030, 3000, 16 * tile - 5, 16), ("adapter", dtype, 16, 600, 1500, 16 * tile - 5, 7),
                  ("adapter", dtype, 24, 600, 130, 6 * tile - 5, 20), ("adapter", dtype, 3, 70, 90, 64, 16),
                  ("adapter", dtype, 2, 1024, 512, 50, 16))
        assert [(v["segments"], bool(v["wide"])) for v in p] == [(4, True), (2, True), (2, False), (1, False), (4, False)]


def test_plans_cover_their_work(plans):
    import random
    rng = random.Random(3)

    def log(hi):
        return min(hi, int(2 ** rng.uniform(0, hi.bit_length())))
    scans, adapters = [], []
    for _ in range(3000):
        G = log(64)
        scans.append(("scan", log(1 << 12), G * log(1 << 12), log((1 << 30) - 1), log(256), G))
        adapters.append(("adapter", rng.randrange(3), log(1 << 12), log(1 << 14), log(1 << 14), log((1 << 24) - 1), log(128)))
    for (_, B, D, L, N, G), p in zip(scans, plans(*scans)):
        chunk = 16 * p["ti"]
        assert p["segments"] * p["chunks"] * chunk >= L > (p["segments"] - 1) * p["chunks"] * chunk
        assert p["groups"] == B * G * -(-(D // G) // 16) and (p["ti"] == 16 or p["segments"] == 1)
        lds = (2 * 16 * chunk + 17 * (N + 1) * 2) * 4
        assert lds <= 65536
    for (_, t, B, C, M, L, R), p in zip(adapters, plans(*adapters)):
        assert p["mtiles"] * p["mrows"] >= M > (p["mtiles"] - 1) * p["mrows"]
        if p["token"]:
            assert p["up"] == B * L * p["mtiles"]
            continue
        tile = 64 if t == 0 else 128
        sets = -(-p["ltiles"] // 4) if p["wide"] else p["ltiles"]
        assert p["ltiles"] * tile >= L > (p["ltiles"] - 1) * tile and p["up"] == B * sets * p["mtiles"]
        assert p["down"] == B * p["ltiles"] * p["segments"] * p["rpieces"] and p["rpieces"] * 64 >= R
        assert (not p["wide"] or R <= 16) and p["mrows"] % 64 == 0


def test_plans_at_the_ends(plans):
    """Under the sanitizer: no sum passes its type."""
    top = (1 << 31) - 1
    conv = plans(("conv", 1, 1, 1, top), ("conv", 0, 7, 1, top), ("conv", 1, 8, 1, top), ("conv", 2, 1, top, 1), ("conv", 0, top, top, top),
                 ("conv", 0, 1, 1, 0))
    assert [p["fits"] for p in conv] == [1, 1, 0, 1, 0, 1] and conv[0]["places"] == 1 << 28 and conv[-1]["places"] == 1
    scan = plans(("scan", 1, top, 1, 1, 1), ("scan", 1, top, 1, 256, top), ("scan", top, 1, 1 << 29, 16, 1), ("scan", 1, 1, (1 << 30) - 1, 16, 1))
    assert [p["fits"] for p in scan] == [0, 0, 0, 1]
    adapter = plans(("adapter", 0, 1, top - 1023, top - 1023, 1, 1), ("adapter", 1, 1, top - 1023, top - 1023, (1 << 30) - 1, 1),
                    ("adapter", 2, top, 1, 1, (1 << 30) - 1, 1), ("adapter", 1, 1, 1, top - 1023, 9, 1))
    assert [p["fits"] for p in adapter] == [1, 0, 0, 1]
