// Token panels of the streamed products (wprod.cuh): how a unit's k's are cut into panels, and which phase of
// its barriers each panel waits for. Plain C++, so that the CPU tests run the same counts.
//
// The panels of a CTA go through kPanels buffers in turn, for all its units one after the other. Per buffer there
// are three mbarriers, each of which completes one phase per use:
//   full    the panel's tokens are in                 used by every panel
//   empty   every multiplying warp has used it        used by every panel
//   landed  they are in, but not yet in pairs         used by the panels that are put into pairs where they lie
// The first two go by the number of panels. Units whose tokens are put into pairs and units whose tokens are not
// may follow each other in one CTA (an expert layer with few and with many assignments to an expert), so `landed`
// has a count of its own.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SIMCOMM_HD __host__ __device__ __forceinline__
#else
#define SIMCOMM_HD inline
#endif

namespace simcomm {

constexpr int kPanelK = 1024;  // a panel: 8 NT tokens x kPanelK / NT k's
constexpr int kPanels = 2;     // buffers

struct PanelCount {
    uint32_t n = 0;      // panels that have gone by, the same for both sides
    uint32_t pairs = 0;  // bit b: the parity of the next phase of landed[b] (the copying warp's side only)
    SIMCOMM_HD int buf() const { return int(n % kPanels); }
    SIMCOMM_HD uint32_t parity() const { return n / kPanels & 1u; }
    SIMCOMM_HD uint32_t landed_parity() const { return pairs >> buf() & 1u; }
    SIMCOMM_HD void used_landed() { pairs ^= 1u << buf(); }  // after the wait for this panel's phase
};

}  // namespace simcomm
