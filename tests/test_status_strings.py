"""A status word that several calls share has a text for every set of device bits."""
import itertools


def test_every_combination_of_device_bits_has_a_text():
    import moe_grouped_gemm_absmax_gb300 as fp8
    names = {fp8.DEV_BAD_OFFSETS: "offsets", fp8.DEV_TIMEOUT: "wait ran out", fp8.DEV_BAD_IDS: "ids"}
    for n in (1, 2, 3):
        for bits in itertools.combinations(names, n):
            text = fp8.status_string(sum(bits))
            assert text.startswith("device:") and all((word in text) == (bit in bits) for bit, word in names.items()), (bits, text)
