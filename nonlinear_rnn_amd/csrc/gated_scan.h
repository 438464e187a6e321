// Gated linear recurrence over time: plan and launches (gated_scan.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace prn {

struct GatedScanArgs {
  bool bf16;                 // storage of every tensor but cu
  int G;                     // 2: [f | v], 3: [f | i | v]
  int64_t B, T, d, n_seqs;   // n_seqs > 0: a ragged pack of T steps (B = 1)
  const int32_t* cu;
  const void *xproj, *h0;    // h0 may be null
  // forward
  void *H, *last;            // last may be null
  // backward (H is read)
  const void *dH, *dlast;    // dlast may be null
  void *dxproj, *dh0;        // dh0 may be null
  unsigned* error;           // device word for a wait that gave up, or null
  unsigned spin_limit;       // polls after which one does
  uint8_t* ws;
  hipStream_t stream;
};

// does the launch fit one grid?
bool gated_scan_fits(const GatedScanArgs& a);
size_t gated_scan_workspace(const GatedScanArgs& a);
void launch_gated_scan(const GatedScanArgs& a);
size_t gated_scan_backward_workspace(const GatedScanArgs& a);
void launch_gated_scan_backward(const GatedScanArgs& a);

}  // namespace prn
