"""The shapes at which the dense products' kernels are tested, by what the library's
plan gives each: the kernel, and the form of its walk or of its join.

PRODUCTS[product][form] are (rows, d_in, d_out) of that product.  Depths pass several
rings of stages, rows and widths end inside a tile.
"""
FEW_BESIDE = {2: 32, 1: 96}   # tokens of a tile up to which the join has a place of its own, by CTAs on an SM

LINEAR_FORMS = {
    "pair, halves": [(4210, 416, 40), (4107, 8, 8)],
    "pair, whole": [(1281, 320, 5000), (10249, 400, 40), (773, 424, 11960)],
    "pair, both": [(843, 400, 9488), (6275, 400, 1288), (9836, 416, 280)],
    "tall, one item": [(4115, 1016, 40)],
    "tall, many items": [(4921, 416, 776), (1300, 1000, 8200), (1500, 2048, 8200)],
    "few, beside, K whole, 1": [(98, 416, 40), (17, 416, 7112)],
    "few, beside, parts, 1": [(17, 440, 2072), (17, 472, 5328), (17, 400, 40), (18, 520, 3360)],
    "few, ring, K whole, 1": [(194, 400, 6368), (100, 408, 9648)],
    "few, ring, parts, 1": [(3883, 1264, 144), (104, 864, 8984), (3685, 2792, 40), (100, 2208, 2848)],
    "few, beside, K whole, 2": [(1, 400, 8216)],
    "few, beside, parts, 2": [(1, 400, 5576), (1, 400, 40)],
    "few, ring, K whole, 2": [(165, 400, 9632)],
}

PRODUCTS = {
    "LINEAR": LINEAR_FORMS,
    "GATED": {
        "pair, halves": [(4210, 416, 40)],
        "pair, whole": [(607, 408, 8048), (10249, 400, 40)],
        "pair, both": [(321, 408, 9504), (9712, 416, 136), (4300, 256, 1096)],
        "tall, one item": [(4115, 1016, 40)],
        "tall, many items": [(130, 400, 9760), (1300, 1000, 5000)],
        "few, beside, K whole, 1": [(98, 416, 40), (17, 408, 3688)],
        "few, beside, parts, 1": [(17, 416, 1072), (17, 464, 2640), (17, 400, 40), (17, 520, 1768)],
        "few, ring, K whole, 1": [(193, 400, 3368), (98, 416, 4848)],
        "few, ring, parts, 1": [(3922, 1360, 72), (97, 848, 4632), (205, 1952, 1000)],
        "few, beside, K whole, 2": [(1, 400, 4128)],
        "few, beside, parts, 2": [(1, 400, 2744), (1, 400, 40)],
        "few, ring, K whole, 2": [(165, 416, 4960), (34, 400, 9624)],
    },
    "HIDDEN_GRAD": {
        "pair, halves": [(4210, 416, 40)],
        "pair, whole": [(773, 424, 11960), (10249, 400, 40), (1061, 952, 3232)],
        "pair, both": [(843, 400, 9488), (6275, 400, 1288), (4300, 256, 1096)],
        "tall, one item": [(4115, 1016, 40)],
        "tall, many items": [(4921, 416, 776), (1300, 1000, 5000)],
        "few, beside, K whole, 1": [(98, 416, 40), (17, 416, 7112)],
        "few, beside, parts, 1": [(17, 440, 2072), (17, 472, 5328), (17, 400, 40)],
        "few, ring, K whole, 1": [(194, 400, 6368), (100, 408, 9648)],
        "few, ring, parts, 1": [(3883, 1264, 144), (104, 864, 8984), (100, 2208, 2848)],
        "few, beside, K whole, 2": [(1, 400, 8216)],
        "few, beside, parts, 2": [(1, 400, 5576), (1, 400, 40)],
        "few, ring, K whole, 2": [(165, 400, 9632)],
    },
    "INPUT_GRAD": {
        "pair, halves": [(4450, 40, 200)],
        "pair, whole": [(499, 7112, 1760), (9521, 40, 200)],
        "pair, both": [(9722, 792, 200), (9803, 272, 200)],
        "tall, one item": [(4141, 40, 488)],
        "tall, many items": [(4834, 816, 216)],
        "few, beside, K whole, 1": [(18, 4776, 200)],
        "few, beside, parts, 1": [(17, 2064, 208), (18, 5304, 200), (17, 40, 200), (17, 2120, 464)],
        "few, ring, K whole, 1": [(233, 6368, 200)],
        "few, ring, parts, 1": [(3780, 136, 616), (99, 5960, 752), (3674, 40, 1360)],
        "few, beside, K whole, 2": [(9, 8264, 136)],
        "few, beside, parts, 2": [(1, 5424, 200), (1, 40, 200)],
        "few, ring, K whole, 2": [(391, 6304, 224)],
    },
    "WEIGHT_GRADS": {
        "pair, halves": [(300, 136, 264)],
        "pair, whole": [(407, 520, 1096)],
        "pair, both": [(129, 6168, 8), (371, 8216, 200)],
    },
}

def form(plan):
    """The name of a plan's form in PRODUCTS."""
    if plan.kernel == "pair":
        return "pair, " + ("both" if plan.tiles and plan.halves else "whole" if plan.tiles else "halves")
    if plan.kernel == "tall":
        return "tall, " + ("one item" if plan.tiles <= 74 else "many items")
    return (f"few, {'beside' if plan.tokens <= FEW_BESIDE[plan.per_sm] else 'ring'}, "
            f"{'K whole' if plan.parts == 1 else 'parts'}, {plan.per_sm}")


def cases(*products):
    return [(rows, d_in, d_out, f) for p in products for f, shapes in PRODUCTS[p].items()
            for rows, d_in, d_out in shapes]
