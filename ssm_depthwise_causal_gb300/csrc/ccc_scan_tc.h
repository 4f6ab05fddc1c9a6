// ccc_scan_tc.h -- arguments and launch interface of the tensor-core scan.
#pragma once

#include <cuda.h>

#include "ccc_scan.h"
#include "ccc_waits.h"

namespace ccc {

struct ScanTcArgs {
    CUtensorMap mv, mk, mc, mo, ms;  // x (or dy), B (or C), C, y: [rows][heads or groups][size], store: boxes of 128 rows of 64
    ScanArgs s;
    int pairs, pairs_per_group, tiles;  // pairs of 64-channel head tiles
    int tail;          // walk only what a cut leaves open
    float *local;      // [parts][128][NW]: an open sequence's state at the CTA's cut
    float *keep;       // [parts][2]: its decay over the CTA's part
    int *flag;         // [parts]: whether that part holds the sequence's start
    float *staged;     // [parts][128][NW]: the slot's state that an open sequence started from
    uint16_t *store;   // [chunk][pair][three parts][128][NW]
    int *status;       // set to 1 when a wait was given up
    Waits waits;
};

// How a call is divided; a function of the host arguments alone.
struct ScanTcPlan {
    bool ok;           // the sizes are the tensor-core kernels'
    int nb, tiles, pairs_per_group, pairs, parts;
    bool cuts;         // whether a cut can fall inside a sequence
    size_t status, local, keep, flag, staged;  // byte offsets in the workspace
    size_t bytes;
};

ScanTcPlan scan_tc_plan(int64_t rows, int n_seqs, int H, int P, int G, int N);

cudaError_t launch_scan_tc_fwd(const ScanArgs &a, const ScanTcPlan &plan, unsigned char *workspace, int *launches, cudaStream_t st);

// A 3-D map of BF16 [rows][count][size] with row stride rs, boxes of box_rows rows of 64, 128-byte swizzle.
bool make_scan_map(CUtensorMap *map, const uint16_t *p, int size, int count, int64_t rows, int64_t rs, int box_rows);

// What each cut leaves open (before launch_walk's kernel, or, `fine`, the states').
cudaError_t launch_scan_tc_tails(ScanTcArgs a, const ScanTcPlan &plan, bool reverse, bool fine, bool first, cudaStream_t st);

// The state before each chunk (reverse: the state gradient after it) into `store`.
cudaError_t launch_scan_tc_states(const ScanArgs &a, const ScanTcPlan &plan, unsigned char *workspace, bool reverse, uint16_t *store,
                                  int *launches, cudaStream_t st);

// What a walk does not meet: the final states (gradient: gradients of initial states) of sequences without rows and padded requests.
cudaError_t launch_edge_states(const ScanArgs &a, float *to, bool gradient, cudaStream_t st);

// The backward's workspace behind the plan's, and its launches.
struct ScanTcBwdPlan {
    ScanTcPlan walk;
    bool ok;
    int heads;   // head tiles
    int64_t slots;
    size_t s_store, g_store, sums, part, bytes;
};

ScanTcBwdPlan scan_tc_bwd_plan(int64_t rows, int n_seqs, int H, int P, int G, int N);

cudaError_t launch_scan_tc_bwd(const ScanArgs &a, const ScanTcBwdPlan &plan, unsigned char *workspace, float *dA, float *dD, float *dbias,
                               int *launches, cudaStream_t st);

}  // namespace ccc
