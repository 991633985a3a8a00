"""Which arrays of a score adjustment's rules are in use (csrc/rules.h), compiled for the host: a rule that is left out takes
its other arrays along, so that the kernel gets no pointer that was not checked."""
import itertools
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "collective_communication_primitives_b200", "csrc")
GROUPS = {"history_len": ("history", "prompt_len", "repetition", "frequency", "presence"), "bias_start": ("bias_token", "bias_value"),
          "mask": ("mask_row",)}
SIZES = {"ld_history": "history_len", "bias_count": "bias_start", "ld_mask": "mask", "mask_rows": "mask"}
ARRAYS = [k for k in GROUPS] + [k for v in GROUPS.values() for k in v]


def test_a_rule_left_out_takes_its_arrays_along(tmp_path):
    lines = ['#include <cstdio>', '#include "rules.h"', 'int main() {', '    static const char wild[1] = {0};']
    for keys in itertools.product((False, True), repeat=3):
        lines.append('    {\n        coll_logit_rules_t u{};')
        for name in ARRAYS:
            if dict(zip(GROUPS, keys)).get(name, True):
                lines.append(f'        u.{name} = reinterpret_cast<decltype(u.{name})>(wild);')
        lines += [f'        u.{name} = 7;' for name in SIZES]
        lines.append('        u = simcomm::rules_in_use(u);')
        lines += [f'        printf("%d ", u.{name} != nullptr);' for name in ARRAYS]
        lines += [f'        printf("%d ", int(u.{name}));' for name in SIZES]
        lines.append('        printf("\\n");\n    }')
    lines.append('    return 0;\n}')
    src, exe = tmp_path / "rules.cpp", tmp_path / "rules"
    src.write_text("\n".join(lines))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    rows = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    for keys, row in zip(itertools.product((False, True), repeat=3), rows, strict=True):
        used = dict(zip(GROUPS, keys))
        want = [int(used[k]) for k in GROUPS] + [int(used[k]) for k, v in GROUPS.items() for _ in v]
        want += [7 if used[k] else 0 for k in SIZES.values()]
        assert [int(v) for v in row.split()] == want, used


def test_the_call_takes_its_rules_from_there():
    with open(os.path.join(CSRC, "api.cu")) as f:
        body = f.read().split("static coll_status_t coll_adjust_logits_impl", 1)[1].split("\n}", 1)[0]
    assert body.count("*rules") == body.count("rules_in_use(*rules)") == 1
    assert "rules->" not in body and "a.rules = u;" in body
