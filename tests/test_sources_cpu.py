"""Rules that the kernels' sources keep, read from the sources."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ATTRIBUTE = re.compile(r"__(launch_bounds|cluster_dims|align)__\((?:[^()]|\([^()]*\))*\)")
FUNCTION = re.compile(r"__(global|device)__[^;{}()]*?(\w+)\(([^{};]*)\)\s*(?:const\s*)?\{", re.S)


def _functions():
    """(file, name, parameters, body, is a kernel) of every function of the kernels' sources."""
    for path in sorted(glob.glob(os.path.join(ROOT, "mla_compressed_latent_b200", "csrc", "*.cu*"))):
        text = ATTRIBUTE.sub("", re.sub(r"//[^\n]*", "", open(path).read()))
        for m in FUNCTION.finditer(text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), m.group(2), m.group(3), text[m.end():i], m.group(1) == "global"


def test_kernels_that_start_early_have_no_restricted_inputs():
    """A kernel that waits for its predecessor, and every device function it calls, takes its inputs without
    restrict: `const T* __restrict__` lets them be loaded through the non-coherent path."""
    functions = list(_functions())
    named = {}
    for f in functions:
        named.setdefault(f[1], []).append(f)
    todo = [f for f in functions if f[4] and "grid_dependency_wait()" in f[3]]
    # (the projection kernels wait in a function they call)
    assert {"append_finish_kernel", "append_fp8_finish_kernel", "read_fp8_kernel", "page_keys_kernel", "select_pages_kernel",
            "merge_kernel", "decode_kernel", "decode8_kernel", "score_kernel", "pair_gemm_kernel", "dequant_pages_kernel",
            "rms_rows_kernel"} <= {f[1] for f in todo}
    seen, bad = set(), []
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.add(f)
        if re.search(r"const \w+\* __restrict__", f[2]) or "__ldg(" in f[3]:
            bad.append(f[:2])
        for name in set(re.findall(r"\b(\w+)(?:<[^;()]*>)?\(", f[3])):
            todo += named.get(name, [])
    assert {"finish_gather", "merge_token_head", "merge_row_quarter"} <= {f[1] for f in seen}
    assert not bad
