"""The token panels of the streamed products (csrc/panels.h), compiled for the host and run against mbarriers of
which every phase is counted: a wait must block until the very phase that its own panel completes. Units that put
their tokens into pairs (up to 8 tokens) and units that do not follow each other in every order, over every number of
panels, as the experts of one call do."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "collective_communication_primitives_b200", "csrc")

PROGRAM = r'''
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include "panels.h"
using namespace simcomm;

// An mbarrier: phase number; a wait with parity P passes once the phase of that parity has completed.
struct Bar {
    uint32_t phase = 0;
    bool passes(uint32_t parity) const { return (phase & 1u) != parity; }
    void complete() { ++phase; }
};

struct Cta {
    Bar full[kPanels], empty[kPanels], landed[kPanels];
    PanelCount copying, multiplying;
    bool one_count;  // the mistake: `landed` waited for by the number of panels

    // The panel of a unit, the copying warp's side, then the multiplying warps'. False at the first wait that does not
    // stand for what the panel itself completes.
    bool panel(bool pairs) {
        const int b = copying.buf();
        if (b != multiplying.buf()) return false;
        if (!empty[b].passes(copying.parity() ^ 1u)) return false;   // its last user has handed it back
        if (full[b].passes(multiplying.parity())) return false;     // nothing is in yet
        if (pairs) {
            const uint32_t parity = one_count ? copying.parity() : copying.landed_parity();
            if (landed[b].passes(parity)) return false;             // the copy is in flight
            landed[b].complete();
            if (!landed[b].passes(parity)) return false;
            copying.used_landed();
        }
        full[b].complete();
        if (!full[b].passes(multiplying.parity())) return false;
        if (empty[b].passes(copying.parity())) return false;        // not handed back yet
        empty[b].complete();
        ++copying.n;
        ++multiplying.n;
        return true;
    }
    bool unit(int nt, int K) {
        for (int k0 = 0; k0 < K; k0 += kPanelK / nt)
            if (!panel(nt == 1)) return false;
        return true;
    }
};

// Units of 1, 2 and 4 token tiles in every order of four, rows of Ka in the first phase and Kb in the second.
static bool holds(int Ka, int Kb, bool one_count) {
    const int tiles[3] = {1, 2, 4};
    for (int order = 0; order < 81; ++order) {
        Cta c;
        c.one_count = one_count;
        for (int phase = 0; phase < 2; ++phase)
            for (int i = 0, o = order; i < 4; ++i, o /= 3)
                if (!c.unit(tiles[o % 3], phase ? Kb : Ka)) return false;
    }
    return true;
}

int main(int argc, char** argv) {
    if (argc > 1 && !std::strcmp(argv[1], "one count")) {  // which rows of K a planted mistake shows at
        for (int K : {512, 1024, 1536, 2048, 2560, 2880, 3584, 4096, 5120, 7168}) std::printf("%d:%d ", K, holds(K, K, true));
        std::printf("\n");
        return 0;
    }
    for (int a = 1; a <= 32; ++a)          // every number of the shortest panels up to 8192 k's, and one with a rest
        for (int b = 1; b <= 32; ++b)
            if (!holds(a * 256, b * 256, false) || !holds(a * 256 - 96, b * 256 - 224, false)) {
                std::printf("FAIL %d %d\n", a, b);
                return 1;
            }
    std::printf("OK\n");
    return 0;
}
'''


def _run(tmp_path, *args):
    src, exe = tmp_path / "panels.cpp", tmp_path / "panels"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe), *args], capture_output=True, text=True)


def test_every_wait_stands_for_its_own_panel(tmp_path):
    res = _run(tmp_path)
    assert res.returncode == 0 and res.stdout.strip() == "OK", res.stdout


def test_one_count_for_both_kinds_of_panels_is_found(tmp_path):
    held = dict(w.split(":") for w in _run(tmp_path, "one count").stdout.split())
    assert [k for k, ok in held.items() if ok == "1"] == ["2048", "4096"], held
