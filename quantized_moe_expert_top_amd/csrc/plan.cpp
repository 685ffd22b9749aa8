// Host-side planning of the launches: which grouped-GEMM kernel runs a call,
// how decode-sized GEMMs split K, and how much workspace each entry point
// needs.  Plain C++: shared by the library and the CPU-only build of the host
// layer, and a pure function of the shapes and the caller's kernel choice
// (the host never reads device counts back).
#include "launch.h"

namespace moe {

// ------------------------------------------------------------- grouping
bool route_permute_fusable(int T, int k, int E) {
  return E <= kRoutePermuteMaxE && (int64_t)T * k <= kPermuteSmallMax;
}

namespace {
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
}  // namespace

// Word 0: invalid-id flag; word 1: arrival counter of the fused routing and
// grouping; then, for the multi-workgroup path, a flag word per chunk and
// the per-chunk key histograms.
size_t permute_workspace_bytes(int P, int E, int S) {
  const size_t nk1 = (size_t)E * S + 1;
  const size_t nb = P <= kPermuteSmallMax ? 0 : (size_t)(P + kPermuteChunk - 1) / kPermuteChunk;
  return 256 + align256(nb * 4) + align256(nb * nk1 * 4);
}

// --------------------------------------------------------------- repack
size_t tiled_salient_bytes(int E, int N, int n_sal) {
  const size_t nsteps = (size_t)(n_sal + 31) / 32;
  return (size_t)E * (N / 16) * nsteps * 1024;
}

// --------------------------------------------------------- grouped GEMM
// K splits of the decode kernel: one unless the (channel group, row tile)
// items leave the chip short of workgroups (fewer than 3 per CU), then enough
// to bring them to about 4 per CU, each split keeping at least 8 K blocks.
int decode_splits(int n_items, int K) {
  const int KBt = K / 128;
  if (n_items >= 768 || KBt < 16) return 1;
  int n = (1024 + n_items - 1) / n_items;
  n = n < KBt / 8 ? n : KBt / 8;
  const int kb_per = (KBt + n - 1) / n;
  return (KBt + kb_per - 1) / kb_per;  // every split non-empty
}

// Upper bound of the decode kernel's row tiles: one partial tile per tile
// segment (an expert, or for MWQ on path 1 each width of an expert).
int decode_row_tiles(int fmt, int path, int M_total, int E) {
  return (M_total + 15) / 16 + ((fmt == 2 && path == 1) ? 3 * E : E);
}

// path: 0 = 16-row tiles (decode kernel; DELTA2: the 32-row delta kernel),
// 1 = 16-row tiles of one width each (nested MWQ), 64 / 65 = 64-row tiles with
// 8 / 4 wavefront columns, 128 = 128-row register-fed tiles, 2 = the 128-row
// LDS-DMA kernel (INT4, nested MWQ; row sums in the workspace), 3 = the
// 128-row LDS-DMA delta kernel (with a shared base, plain epilogues), 5 = the
// LDS-DMA kernel on row tiles of one width each (nested MWQ).
//
// MOE_KERNEL_AUTO chooses from the mean rows per segment (the host never sees
// the device counts): few rows -> 16-row tiles (decode kernel); many -> the
// 128-row LDS-DMA kernel for INT4, 64-row tiles otherwise (and for INT4
// segments of under ~96 rows, where 128-row tiles would be mostly padding),
// with 8 wavefront columns (activations re-read half as often) when the
// activations outweigh the weights, else 4.  Nested MWQ -> from about 24 rows
// per width sub-segment the LDS-DMA kernel on row tiles of one width each
// (measured on the Mixtral-shaped layer at 512 tokens, ~43 rows per
// sub-segment: 447 us for gate/up against 595 us for 16-row chunks of all
// widths per workgroup, whose per-row-tile width masks cost 4 VALU operations
// per MFMA); fewer rows -> 16-row tiles that take all widths of an expert
// together (one read of each bit plane).  Any other MOE_KERNEL_* value is
// taken as given.
int pick_path(const QWeights& w, int M_total, int nseg, int epi, int kernel) {
  const int fmt = w.fmt;
  switch (kernel) {
    case 1: return 0;
    case 2: return 1;
    case 3: return 64;
    case 4: return 65;
    case 5: return 128;
    case 6: return fmt == 3 ? 3 : 2;
    case 7: return 5;
    default: break;
  }
  if (fmt == 4) return 0;  // a width per expert: 16-row tiles at every batch size
  const double avg = (double)M_total / (double)(nseg > 0 ? nseg : 1);
  if (fmt == 3) return (avg >= 96.0 && w.base && epi != 1) ? 3 : 0;
  if (avg < 24.0) return 0;
  if (fmt == 2) return 5;
  if (fmt == 1 && avg >= 96.0) return 2;
  const int E = fmt == 2 ? nseg / 3 : nseg;
  const double a_bytes = (double)M_total * w.K * 2.0;
  const double w_bytes = (double)E * w.N * w.K * (fmt == 1 ? 0.5 : 0.25);
  return a_bytes < w_bytes ? 65 : 64;
}

bool qgemm_kernel_supported(int fmt, int kernel) {
  switch (kernel) {
    case 0: case 1: return true;
    case 2: return fmt == 2;
    case 3: case 4: case 5: return fmt == 1 || fmt == 2;
    case 6: return fmt == 1 || fmt == 2 || fmt == 3;
    case 7: return fmt == 2;
    default: return false;
  }
}

namespace {
size_t ws_need(const QWeights& w, int path, int epi, int A_rows, int M_total) {
  if (path == 2 || path == 5) return ((size_t)A_rows * (w.K / w.G) * 4 + 255) & ~(size_t)255;  // row sums per group
  if (path == 3) return ((size_t)A_rows * 4 + 255) & ~(size_t)255;                 // row sums over all of K
  if (w.fmt != 3 && epi != 1 && (path == 0 || path == 1)) {
    // split-K partial sums of the plain epilogues (the SwiGLU one never splits)
    const int n_ks = decode_splits(((w.N + 127) / 128) * decode_row_tiles(w.fmt, path, M_total, w.E), w.K);
    if (n_ks > 1) return ((size_t)n_ks * M_total * w.N * 4 + 255) & ~(size_t)255;
  }
  return 0;
}
}  // namespace

size_t qgemm_workspace_bytes(const QWeights& w, int A_rows, int M_total, int kernel) {
  const int nseg = w.E * (w.fmt == 2 ? 3 : 1);
  size_t need = 0;
  for (int epi = 0; epi < 4; ++epi) {
    const size_t n = ws_need(w, pick_path(w, M_total, nseg, epi, kernel), epi, A_rows, M_total);
    need = n > need ? n : need;
  }
  return need;
}

// The start of an MX layer counts its pairs while every workgroup of the second
// launch can read all counts (E + 1 per chunk of a workgroup's tokens): up to
// 256 K of them, or 3 per pair and 1.1 M; with more, grouping is a call of its
// own.  Layers of 128 x 128 experts, us so / apart: 64 experts 74 / 87 (16384
// tokens x 8, 67 K counts), 502 / 611 (131072, 532 K); 256 experts 362 / 383
// (65536 x 8, 1.05 M); 1000 experts 48 / 65 (1000 x 4, 125 K), 66 / 67 (2048,
// 256 K), 91 / 79 (4096, 512 K).
int front_chunk_tokens(int T, int k, int E) {
  const int tokens = chunk_tokens((E + 63) / 64);
  const int64_t counts = ((int64_t)T + tokens - 1) / tokens * (E + 1);
  const int64_t by_pairs = 3 * (int64_t)T * k < 1100 * 1024 ? 3 * (int64_t)T * k : 1100 * 1024;
  return counts <= 256 * 1024 || counts <= by_pairs ? tokens : 0;
}
size_t mx_layer_workspace_bytes(int T, int k, int E) {
  const size_t sort = permute_workspace_bytes(T * k, E, 1);
  const int tokens = front_chunk_tokens(T, k, E);
  if (tokens == 0) return sort;
  const size_t counts = 256 + align256((size_t)(T + tokens - 1) / tokens * (E + 1) * 4);
  return counts > sort ? counts : sort;
}

// Grouped MX product: 0 = 32-row tiles straight from memory, 64 / 128 =
// LDS-staged tiles of that many rows.  AUTO takes the least of three estimates
//     a + K * max(b, c * (workgroups / 256 + d))      (microseconds)
// a: launch and set-up, b: one workgroup alone on its CU, c: a CU's throughput,
// d: its last workgroups running alone.  Fitted to 346 measured problems (E 8 to
// 64, 1 to 1024 rows per expert, N 448 to 28672, K 512 to 14336, 8- and 4-bit
// rows alike) with weights that stay in the cache where they fit, and before the
// kernels' last changes.  They rank the paths rather than tell the time: over 260
// problems with weights from memory four in five times are 0.72 to 1.45 of the
// estimate (all 0.59 to 1.94), the path taken 1.3 % above the best of all on average,
// over 10 % in 10 of them, 33 % at most (8 experts of 2048 x 2048, 32 e2m1 rows each:
// 12.0 for 9.0 us).  E.g. 8 experts of 2048 x 2048, e4m3 rows, us for 32-row / 64-row /
// 128-row tiles: 8.4 / 11.2 / 11.0 at 16 rows per expert, 18.8 / 12.2 / 17.5 at 128; 64
// experts at 512 rows: 453 / 134 / 126.
// 64-row tiles of e2m1 rows split K over two groups of wavefronts where K is long
// and every workgroup has a CU of its own: 8 experts of 4096 x 14336, 32 rows each
// 72 -> 65 us, 16 of 448 x 4096, 192 rows 18.6 -> 17.4; with K = 2048 11.9 both, with
// 768 workgroups 48 -> 58.  With e4m3 rows, whose stages hold twice the bytes, the
// split lost (15.4 -> 16.2).
int mxgemm_path(int M_total, int E, int N, int K, bool e2m1, int kernel) {
  if (kernel == 1) return 0;
  const double active = M_total < E ? M_total : E;  // experts that can have rows
  const double nt = N / 32.0;
  const double wide_blocks = (double)(int64_t)((nt + 7.0) / 8.0);
  const int path64 = e2m1 && K >= 4096 && wide_blocks * (M_total / 64.0 + 0.5 * active) <= 256.0 ? kMxSplit : 64;
  if (kernel == 4) return 64;
  if (kernel == 8) return kMxSplit;
  if (kernel == 5) return 128;
  int best = 0;
  double least = 0.0;
  const int rows[3] = {32, 64, 128}, path[3] = {0, path64, 128};
  const double a[3] = {2.6, 2.7, 3.8}, b[3] = {1.2e-3, 3.0e-3, 3.0e-3}, c[3] = {1.71e-3, 4.0e-3, 6.9e-3},
               d[3] = {0.5, 0.5, 0.4};
  // the partial tile per expert, and its least work: fewer rows take a smaller body
  const double partial[3] = {0.5, 0.4, 0.125}, fewest[3] = {1.0, 1.0, 0.5};
  for (int i = 0; i < 3; ++i) {
    double tiles = (double)M_total / rows[i] + partial[i] * active;
    if (tiles < fewest[i] * active) tiles = fewest[i] * active;
    const double wide = i == 0 ? 2.0 : 8.0;  // channel tiles of a workgroup
    const double blocks = (nt + wide - 1.0) / wide;
    // 32-row tiles read only the rows there are
    const double fill = i == 0 && M_total < 32.0 * active ? 0.62 + 0.38 * M_total / (32.0 * active) : 1.0;
    const double cu = fill * c[i] * (tiles * (double)(int64_t)blocks / 256.0 + d[i]);
    const double t = a[i] + K * (cu > b[i] ? cu : b[i]);
    if (i == 0 || t < least) {
      least = t;
      best = path[i];
    }
  }
  return best;
}

}  // namespace moe
