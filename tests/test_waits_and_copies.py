"""How the kernels' bounded waits end, read from the sources (no GPU needed): a CTA
whose copies may still be in flight after a wait that gave up lets them land before
it ends, since its shared memory may belong to another CTA by the time they do."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_quantized_matmul_b200", "csrc")


def _code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


def _functions(src):
    """{name: (is a kernel, body)} of the functions at namespace level."""
    out = {}
    for h in re.finditer(r"(__global__|__device__)[^;{}]*?\b(\w+)\s*\((?!\s*\d)[^;{}]*\)\s*\{", src):
        depth, i = 1, h.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        head = re.sub(r"__launch_bounds__\([^)]*(\([^)]*\)[^)]*)*\)", "", h.group(0))
        name = re.search(r"(\w+)\s*\(", head).group(1)
        out[name] = (h.group(1) == "__global__", src[h.end():i])
    return out


def _reach(functions, name, seen):
    body = functions[name][1]
    seen.add(name)
    for other in functions:
        if other not in seen and re.search(rf"\b{other}\s*[(<]", body):
            body += _reach(functions, other, seen)
    return body


KERNELS = [("adapter.cu", "tile_shrink_kernel"), ("adapter.cu", "tile_expand_kernel"), ("scaled_matmul.cu", "weight_stream_kernel"),
           ("gemm_sm100.cu", "gemm_i8_persistent_kernel"), ("gemm_groups.cu", "gemm_groups_kernel"), ("decode.cu", "decode_kernel")]


def test_the_list_has_every_kernel_that_copies_tiles():
    found = set()
    for f in sorted(os.listdir(CSRC)):
        if f.endswith(".cu"):
            functions = _functions(_code(f))
            found |= {(f, k) for k, (kernel, _) in functions.items()
                      if kernel and "tma_load_" in _reach(functions, k, set())}
    assert found == set(KERNELS)


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_copies_land_after_a_wait_that_gave_up(file, kernel):
    body = _functions(_code(file))[kernel][1]
    # before tensor memory is given back, and with nothing but the CTA's last barrier near it
    land, free = body.rfind("let_copies_land()"), body.rindex("tmem_dealloc")
    assert land != -1, "ends with copies in flight"
    assert land < free and abs(body.rindex("__syncthreads()") - land) < 60


def test_partial_sums_do_not_overwrite_a_ring_that_copies_still_go_to():
    body = _functions(_code("scaled_matmul.cu"))["weight_stream_kernel"][1]
    first = body.find("let_copies_land()")
    assert -1 < first < body.index("part[(c + i) * kRows")


def test_the_product_gives_up_as_one():
    """Every wait of the product's kernel watches the flag that the first to give up raises."""
    body = _functions(_code("scaled_matmul.cu"))["weight_stream_kernel"][1]
    assert not re.search(r"\bmbar_wait\(", body) and body.count("wait_or_give_up(") == 4
