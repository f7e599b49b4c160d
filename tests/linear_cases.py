"""Shapes of linear layers by the kernel that the library's plan gives them (no code
of the package)."""
import torch

F32, BF16 = torch.float32, torch.bfloat16

# (x's type, the list's, input gradient) -> {(tile, sliced, parts or copies made beforehand of A, of B): (rows, out, in)}.
# Tile 0, 1, 2 as the plan numbers them, -1 for few tokens on the vector units; sizes end inside tiles, 32-row blocks and steps.
PLANS = {
    (BF16, BF16, False): {
        (0, False, 0, 0): (3384, 2414, 488), (0, False, 1, 1): (1705, 5011, 454), (0, True, 0, 0): (1030, 3600, 3080),
        (0, True, 1, 1): (1041, 3625, 3143), (1, False, 0, 0): (3482, 537, 40), (1, False, 1, 1): (4248, 411, 39),
        (1, True, 0, 0): (1384, 166, 1936), (1, True, 1, 1): (1375, 149, 1935), (2, False, 0, 0): (75, 141, 48),
        (2, False, 1, 1): (76, 154, 38), (2, True, 0, 0): (84, 143, 728), (2, True, 1, 1): (71, 190, 741)},
    (BF16, BF16, True): {
        (0, False, 0, 0): (2391, 456, 3336), (0, False, 0, 1): (4854, 526, 2128), (0, False, 1, 0): (3949, 680, 2074),
        (0, False, 1, 1): (1871, 449, 4673), (0, True, 0, 0): (1030, 3080, 3600), (0, True, 1, 0): (3100, 3080, 1290),
        (1, False, 0, 0): (4346, 48, 392), (1, False, 1, 1): (4179, 41, 385), (1, True, 0, 0): (1383, 1720, 264),
        (1, True, 0, 1): (1441, 1812, 304), (1, True, 1, 1): (1130, 2107, 287), (2, False, 0, 0): (87, 40, 152),
        (2, False, 1, 1): (80, 37, 141), (2, True, 0, 0): (71, 712, 168), (2, True, 1, 1): (79, 709, 151)},
    (BF16, F32, False): {
        (0, False, 1, 0): (3100, 1290, 136), (0, False, 1, 1): (4303, 385, 292), (0, True, 1, 1): (776, 775, 1539),
        (1, False, 1, 1): (73, 151, 37), (1, True, 1, 1): (78, 152, 412), (2, False, 0, 0): (74, 141, 40),
        (2, True, 0, 0): (75, 161, 208), (2, True, 0, 1): (75, 270, 777)},
    (BF16, F32, True): {
        (0, False, 1, 1): (1718, 317, 1177), (0, True, 1, 0): (1117, 1456, 520), (1, False, 1, 1): (70, 33, 174),
        (1, True, 1, 1): (80, 363, 158), (2, False, 0, 0): (70, 48, 144), (2, True, 0, 0): (72, 208, 184)},
    (F32, BF16, False): {
        (0, False, 0, 1): (1315, 1636, 296), (0, True, 1, 1): (930, 780, 1255), (1, False, 1, 1): (91, 143, 34),
        (1, True, 1, 1): (74, 150, 355), (2, False, 0, 0): (78, 163, 40), (2, True, 0, 0): (73, 157, 200),
        (2, True, 1, 0): (300, 40, 777)},
    (F32, BF16, True): {
        (0, False, 0, 1): (1036, 295, 2072), (0, False, 1, 1): (1036, 295, 1971), (0, True, 1, 1): (566, 1466, 1210),
        (1, False, 1, 1): (76, 35, 156), (1, True, 1, 1): (81, 365, 187), (2, False, 0, 0): (77, 40, 152),
        (2, True, 0, 0): (71, 248, 144)},
    (F32, F32, False): {
        (0, False, 1, 1): (1479, 1286, 136), (0, True, 1, 1): (668, 923, 1040), (1, False, 1, 1): (787, 779, 344),
        (1, True, 1, 1): (972, 664, 880), (2, False, 0, 0): (83, 141, 34), (2, True, 0, 0): (88, 142, 131)},
    (F32, F32, True): {
        (0, False, 1, 1): (2051, 138, 933), (0, True, 1, 1): (936, 1093, 724), (1, False, 1, 1): (984, 347, 646),
        (1, True, 1, 1): (654, 888, 920), (2, False, 0, 0): (72, 33, 145), (2, True, 0, 0): (84, 134, 145)},
}
FEW = {False: [(1, 141, 1032), (3, 141, 2600), (8, 4101, 1032), (4, 4101, 2056), (7, 30, 70)],
       True: [(1, 1032, 141), (3, 4100, 141), (8, 2600, 141), (5, 700, 333)]}


def shapes(parts_only=False):
    """(x's type, the list's, input gradient, rows, out, in) of every entry; parts_only: where an fp32 operand is cut."""
    out = []
    for (xt, lt, back), by in PLANS.items():
        if not parts_only or F32 in (xt, lt):
            out += [(xt, lt, back, *s) for s in by.values()]
    if not parts_only:
        out += [(xt, lt, back, *s) for xt, lt, back in PLANS for s in FEW[back]]
    return out


def name(case):
    xt, lt, back, rows, out, inp = case
    short = {F32: "f32", BF16: "bf16"}
    return f"{'grad' if back else 'forward'}-{short[xt]}-{short[lt]}-{rows}-{out}-{inp}"
