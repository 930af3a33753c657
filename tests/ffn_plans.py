"""Sizes of the feed-forward block that between them run every way in which its products may be
launched: tile, rows of the first operand's boxes, results that leave at once or as parts, for
sizes of vectors and odd ones."""
import ctypes

import chunked_prefill_gdn_gb300 as gdn

SHAPES = {"bf16": [
    (17, 17, 11, 10), (17, 712, 2784, 16), (17, 1232, 1000, 72), (17, 3784, 16, 24), (18, 695, 2771, 86),
    (18, 1220, 11, 14), (18, 4332, 10, 963), (22, 959, 748, 213), (27, 200, 7192, 64), (32, 16, 16, 16),
    (33, 1117, 930, 62), (33, 2424, 40, 224), (33, 4142, 9, 108), (35, 29, 2376, 79), (46, 1152, 928, 32),
    (47, 16, 3200, 24), (47, 776, 592, 80), (58, 5128, 3416, 64), (65, 64, 6232, 3304), (65, 2280, 24, 48),
    (66, 16, 2288, 120), (67, 2868, 9, 144), (69, 11, 6708, 3365), (77, 3762, 3262, 29), (84, 19, 1285, 85),
    (98, 148, 6914, 42), (129, 560, 4968, 3592), (130, 408, 2508, 519), (133, 447, 5977, 2786), (135, 2826, 3022, 83),
    (140, 4776, 1744, 48), (291, 760, 1928, 32), (1075, 24, 8808, 16), (1445, 16, 1568, 16), (1572, 136, 1432, 176),
    (1735, 136, 1383, 232), (1751, 136, 1552, 64), (2349, 14, 4569, 10), (2480, 14, 3140, 13), (2884, 132, 957, 12),
    (3250, 26, 682, 13), (3285, 40, 1328, 16), (3435, 32, 2912, 16), (4893, 20, 770, 28), (5351, 32, 136, 1528)],
          "f32": [
    (10, 16, 6256, 24), (12, 48, 5888, 24), (13, 16, 6115, 14), (19, 21, 6444, 15), (36, 5112, 80, 5168),
    (38, 16, 16, 16), (40, 16, 7616, 792), (51, 9, 13, 12), (54, 88, 456, 32), (62, 138, 3767, 9), (92, 97, 631, 11),
    (133, 28, 1582, 1289), (133, 496, 8520, 264), (159, 216, 3144, 32), (198, 72, 352, 40), (210, 32, 200, 24),
    (222, 25, 237, 11), (258, 5935, 9, 14), (261, 40, 9872, 1440), (264, 20, 2089, 9), (268, 55, 11001, 945),
    (279, 468, 4109, 394), (282, 1192, 208, 664), (288, 82, 6430, 1750), (330, 155, 1932, 11), (350, 24, 16, 16),
    (373, 56, 6592, 1504), (418, 5348, 65, 50), (426, 9, 10, 9), (449, 3152, 136, 5184), (523, 152, 1048, 40),
    (937, 16, 72, 5208), (1033, 60, 66, 4532), (1364, 216, 264, 104), (1495, 14, 3196, 573), (1900, 288, 688, 16),
    (2305, 293, 586, 28), (2528, 202, 205, 23), (7304, 88, 560, 768), (7664, 9, 158, 314)]}


def plan(lib, M, D, F, O, dtype, backward):
    p = ctypes.c_void_p(4096)   # aligned; never dereferenced
    d = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, D, M, D, F, O, 0, 1 if dtype == "f32" else 0)
    info = gdn.GdnFfnPlanInfo()
    assert lib.gdn_gated_ffn_plan_query(d, backward, p, O, info) == 0
    return info


def ways(lib, M, D, F, O, dtype):
    """How the launches of a forward and a backward pass run.  Of the four gradients: all at
    once, all as parts or some of each, and whether a part of dx runs from one pair of operands
    into the other (an odd number of parts)."""
    out = set()
    vectors = D % 8 == F % 8 == O % 8 == 0
    for backward, names in ((0, ("up", "y")), (1, ("dh", "gradients"))):
        info = plan(lib, M, D, F, O, dtype, backward)
        if info.path != 2:
            continue
        for i, name in enumerate(names):
            parts = list(info.parts[i])[:info.products[i]]
            cut = name == "gradients" and parts[0] > 1 and parts[0] % 2 == 1
            state = "at once" if not any(parts) else "parts" if all(parts) else "some parts"
            out.add((name, dtype, info.tile[i], info.a_rows[i], state, cut, vectors))
    return out
