// Library-internal declarations shared by the HIP translation units of libosc.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "osc.h"

namespace osc {

// Table slice passed by value in the kernel arguments: the per-layer row of the
// offline table lives in the kernarg segment for the duration of the launch.
struct TableArg {
  int8_t v[OSC_MAX_GROUPS];
};

enum TableMode { kNoTable = 0, kExtractZero = 1, kCopyOnly = 2 };

// Most protected channels per group the kernels handle (m = 1 is the single-channel method).
constexpr int kMaxChannels = 3;

// Quantize rows of a bf16 matrix in groups of G (activations or weights); the table holds m
// entries per group, entry e of group k at v[k*m + e].
//   mode kExtractZero: B(r, k*m+e) <- X[r][kG+L[k][e]], those slots are zeroed before scaling.
//   mode kCopyOnly:    WL(r, k*m+e) <- W[r][kG+L[k][e]], nothing is zeroed.
// glu: X holds rows of 2H bf16 (gate | up) and the row quantized is h = silu(gate) * up
// (binary32, rounded to bf16), the input of a gated MLP's down-projection.
hipError_t launch_quant(const void* X, int rows, int H, int G, int m, const TableArg* tab, int mode, osc_fmt fmt,
                        void* Q, uint8_t* SC, void* side, hipStream_t st, bool glu = false);

// h = silu(gate) * up (the same binary32 definition as the glu quantization), written as bf16:
// GU rows of 2F bf16 -> Hout rows of F bf16.
hipError_t launch_swiglu(const void* GU, int rows, int F, void* Hout, hipStream_t st);

// Table slice with up to m entries per group: L and hits device int32[K*m], events int32[K].
hipError_t launch_build_table(const void* Xcal, int R, int H, int G, int m, double alpha, double rho, int32_t* L,
                              int32_t* hits, int32_t* events, hipStream_t st);

struct GemmArgs {
  const void* QX;
  const uint8_t* SX;
  const void* B;
  const void* QW;
  const uint8_t* SW;
  const void* WL;
  void* Y;
  int S, N, H, G;
  int kc;  // compensation columns (m*K), 0 without compensation
  osc_fmt afmt, wfmt;
  osc_ytype yt;
};

hipError_t launch_gemm(const GemmArgs& a, hipStream_t st);

// The prefill GEMMs' XCD tile blocks for a grid of ntm x ntn tiles of BM x BN (the kernels'
// xblk argument; see xcd_tile in osc_device.h).
int xcd_blocks(int ntm, int ntn, int BM, int BN);

// MXFP4 activations and weights at G = 32 / 64, E4M3 activations with MXFP4 weights (the W2
// fallback) and the E3M2 pairs, on 32x32 scaled MFMA blocks (the prefill path of launch_gemm for
// those formats).
hipError_t launch_gemm_mx4(const GemmArgs& a, hipStream_t st);

// S <= 32 rows: the skinny-S kernel (one 32-column block per workgroup, K split over its waves).
constexpr int kDecodeRows = 32;
hipError_t launch_gemm_dec(const GemmArgs& a, hipStream_t st);

// S <= 32 rows with the activation quantization fused into the skinny-S GEMM (MXFP4 both sides):
// X [S][H] bf16 row-major, the table (or none: WL == nullptr), the packed weights.
struct FusedArgs {
  const void* X;
  const TableArg* tab;
  int m;
  const void* QW;
  const uint8_t* SW;
  const void* WL;
  void* Y;
  int S, N, H, G;
  int kc;  // compensation columns (m*K), 0 without compensation
  osc_ytype yt;
};
// LDS bytes the fused kernel needs for this shape (the limit is 160 KiB per workgroup).
long fused_lds_bytes(int H, int G, int kc);
hipError_t launch_linear_dec(const FusedArgs& a, hipStream_t st);

// What lies between the projections.  The functions are weak references: a library linked from the linear layers'
// objects alone (the sanitizer build of the validation) loads and checks every argument, and answers OSC_E_DEVICE
// where it would launch.
#define OSC_STEP __attribute__((weak))

// Residual add + RMS norm of S rows of H bf16; SX == nullptr: y itself to QX (row-major bf16), else its
// quantization, tab == nullptr without extraction.
struct NormArgs {
  const void *X, *RES, *W;
  int S, H;
  float eps;
  int G, m;
  const TableArg* tab;
  osc_fmt afmt;
  void* RES_OUT;
  void* QX;
  uint8_t* SX;
  void* B;
};
OSC_STEP hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st);

// Page tables and slot maps of one step (osc_page_plan); sh = log2(page).
struct PlanArgs {
  const int32_t *CTX, *NEW;
  int R, sh, NP;
  const int32_t* FREE;
  int F;
  const int32_t* HEAD;
  int T;
  int32_t* TABLE;
  int MB;
  int32_t *CU, *KV, *SLOT, *POS, *USED;
};
OSC_STEP hipError_t launch_page_plan(const PlanArgs& a, hipStream_t st);

// Head norm, rotary embedding and cache write (osc_qkv_append); sh = log2(page).
struct AppendArgs {
  const void* QKV;
  int S, HQ, HKV, D;
  const void *WQ, *WK;
  float eps;
  const float* CS;
  int P;
  const int32_t *POS, *SLOT;
  void *Q, *KC, *VC;
  int NP, sh;
};
OSC_STEP hipError_t launch_qkv_append(const AppendArgs& a, hipStream_t st);

// Attention over the paged cache (osc_attn_paged).
struct AttnPlan {
  bool small;       // 16-row tiles
  int target;       // workgroups for each key head that cut tiles are dealt to (0: none is cut)
  int grid;         // workgroups for each key head
  long ws_bytes;
};
OSC_STEP AttnPlan attn_plan(int S, int R, int HQ, int HKV, int D, long keys);  // keys: of a table's row
struct AttnArgs {
  const void *Q, *KC, *VC;
  int S, R, HQ, HKV, g;  // g = HQ / HKV
  int sh, mask, MB, NP;  // page = 1 << sh, mask = page - 1
  const int32_t *TABLE, *CU, *KV;
  float scale_log2;  // scale * log2(e)
  void* O;
  // Workspace, where tiles are cut: [HKV][target] notes of the workgroups; [HKV][target][2 places][rows of a tile]
  // scaled maximum and sum, and D unnormalised outputs.
  float* PO;
  float* PM;
  int4* NOTE;
  int target;
};
OSC_STEP hipError_t launch_attn(const AttnArgs& a, int D, const AttnPlan& p, hipStream_t st);

// Attention with a mask among a request's new tokens (osc_attn_tree): MASK [S][W].
struct TreePlan {
  int N;         // nodes of a tree, at most
  int rows;      // of a tile: 16 or 256
  int target;    // workgroups for each key head
  long ws_bytes;
};
OSC_STEP TreePlan attn_tree_plan(int HQ, int HKV, int D, int N);
struct TreeArgs : AttnArgs {
  const unsigned long long* MASK;
  int W;
};
OSC_STEP hipError_t launch_attn_tree(const TreeArgs& a, int D, const TreePlan& p, hipStream_t st);

// Log probabilities (osc_logprobs); rows are cut into `chunks` parts where there are few.
struct LogprobsPlan {
  int chunks;
  long ws_bytes;
};
OSC_STEP LogprobsPlan logprobs_plan(int S, int V, int K);
struct LogprobsArgs {
  const void* X;
  osc_ytype xt;
  int S, V, ld;
  float scale_log2;  // scale * log2(e)
  const int32_t* ID;
  int M, K;
  float *LP, *ENT, *TOPV;
  int32_t* TOPI;
  void* WS;
  int chunks;
};
OSC_STEP hipError_t launch_logprobs(const LogprobsArgs& a, hipStream_t st);

// Token trees (osc_tree_plan, osc_tree_accept, osc_tree_commit).
struct TreeMaskArgs {
  const int32_t *PARENT, *CU, *CTX;
  int R, T, N, W;
  int32_t* POS;
  unsigned long long* MASK;
};
OSC_STEP hipError_t launch_tree_plan(const TreeMaskArgs& a, hipStream_t st);
struct AcceptArgs {
  const int32_t *TOKEN, *PARENT, *CHOICE;
  int ldc;
  const int32_t *SLOT, *POS;
  int P;
  const int32_t* CU;
  int R, T, N;
  int32_t *ACC, *PATH, *NEXT;
};
OSC_STEP hipError_t launch_tree_accept(const AcceptArgs& a, hipStream_t st);
struct CommitArgs {  // by value: the pointers travel in the kernel's arguments
  void* KC[OSC_MAX_LAYERS];
  void* VC[OSC_MAX_LAYERS];
  int layers, NP, HKV, D, sh;
  const int32_t *SLOT, *CU, *ACC, *PATH;
  int R, T, N;
};
OSC_STEP hipError_t launch_tree_commit(const CommitArgs& a, hipStream_t st);

}  // namespace osc
