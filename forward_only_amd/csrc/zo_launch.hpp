// zo_launch.hpp -- host-side launchers of the gfx950 kernels (internal to libzo).
// Arguments are validated by the C ABI layer (api.hip) before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zo {

struct Key {
    uint32_t k0, k1;  // Philox key = (seed_lo, seed_hi)
};

// Packed sign rows: rows of ceil(n/128)*16 bytes for probes probe0 .. probe0+nprobes-1.
hipError_t launch_gen_probes(Key key, uint32_t step, uint32_t probe0, uint32_t nprobes,
                             uint64_t offset, uint64_t n, uint8_t *bits, int num_cus,
                             hipStream_t stream);

// Slice lengths of the perturb passes are multiples of this many params (a whole number of
// the kernel's chunks: 4096 bf16 or 2048 fp32 params, 8 KiB each).
constexpr uint64_t kPerturbChunkParams = 4096;

// Workgroups of a non-persistent XCD-range launch (xcd_range_chunk) over n chunks with
// `waves` waves per workgroup: eight times those of the longest range (ranges differ by at
// most one chunk, so the longest holds ceil(n / 8)).  Launches cover at most
// kMaxChunksPerLaunch chunks, which keeps the grid below 2^31 workgroups even with one wave
// per workgroup.
constexpr uint64_t kMaxChunksPerLaunch = (uint64_t)1 << 30;
inline uint32_t xcd_range_grid(uint64_t n, uint32_t waves)
{
    return (uint32_t)(8 * (((n + 7) / 8 + waves - 1) / waves));
}

// theta[0..n) += alpha * z (fp32 or bf16), bits == nullptr regenerates.  slice > 0 (a
// multiple of kPerturbChunkParams) issues the pass as one launch per slice of that many
// params; 0 is one launch.
hipError_t launch_perturb(void *theta, bool bf16, uint64_t offset, uint64_t n, Key key,
                          uint32_t step, uint32_t probe, float alpha, const uint8_t *bits,
                          int num_cus, hipStream_t stream, uint64_t slice = 0);

// theta[0..n) += (+/-alpha_a) + (+/-alpha_b) in one pass (probes a and b); bits_a and
// bits_b are both given or both nullptr.  slice as launch_perturb.
hipError_t launch_perturb2(void *theta, bool bf16, uint64_t offset, uint64_t n, Key key,
                           uint32_t step, uint32_t probe_a, float alpha_a, uint32_t probe_b,
                           float alpha_b, const uint8_t *bits_a, const uint8_t *bits_b,
                           int num_cus, hipStream_t stream, uint64_t slice = 0);

// c[i] from (L+, L-, L0) in fp64; non-finite probes counted into *counter.
// mode 0: g / max(|h|, delta); 1: g / max(|h|, delta)^power; 2: g / npert (L0 unused).
hipError_t launch_probe_weights(const double *Lp, const double *Lm, const double *L0,
                                uint32_t npert, double eps, double delta, int mode,
                                double power, float *c, uint32_t *counter, hipStream_t stream);

// Largest probe count of one update (its sign tables live in LDS).
constexpr uint32_t kMaxNpert = 512;

// Raise the dynamic-LDS limit of the general update kernels to what kMaxNpert needs, on the
// current device (once per context, from zo_init; launches then call no attribute setter).
hipError_t prepare_update();

// theta[0..n) -= eta * sum_i c_i z_i through per-8-probe LDS tables.
hipError_t launch_update(void *theta, bool bf16, uint64_t offset, uint64_t n, Key key,
                         uint32_t step, const float *c, uint32_t npert, float eta,
                         const uint8_t *bits, int num_cus, hipStream_t stream);
// The update preceded, in the same pass, by the move theta + alpha_r * z_rprobe rounded as
// launch_perturb rounds it (rprobe < npert).
hipError_t launch_restore_update(void *theta, bool bf16, uint64_t offset, uint64_t n, Key key,
                                 uint32_t step, uint32_t rprobe, float ralpha, const float *c,
                                 uint32_t npert, float eta, const uint8_t *bits, int num_cus,
                                 hipStream_t stream);

// counter[0] = 0 with a fill kernel (no memset node if the caller captures a graph).
hipError_t launch_zero_u32(uint32_t *p, uint32_t count, hipStream_t stream);

// 1/2 sum a_j theta_j^2 in fp64, two deterministic passes through `partials`.
constexpr uint32_t kLossPartials = 1024;
hipError_t launch_quad_loss(const void *theta, bool bf16, const float *a, uint64_t n,
                            double *partials, double *out, hipStream_t stream);
constexpr uint32_t kQuadProbes = 4;   // probes per pass of the fused quadratic losses
// The same loss at theta +/- alpha z_i for n_probes consecutive probes from probe0, theta
// read once per kQuadProbes probes and never written; each loss bit-equal to zo_perturb
// followed by launch_quad_loss.  With out_clean the first pass also sums the loss at theta
// itself, bit-equal to launch_quad_loss.  `partials` as for launch_quad_loss (2 kQuadProbes
// + 1 slots).
hipError_t launch_quad_loss_probes(const void *theta, bool bf16, const float *a, uint64_t offset,
                                   uint64_t n, Key key, uint32_t step, uint32_t probe0,
                                   uint32_t nprobes, float alpha, const uint8_t *bits,
                                   double *partials, double *out_plus, double *out_minus,
                                   double *out_clean, hipStream_t stream);

// 1/2 sum a_j theta_j^2 + 1/2 ||U theta||^2, U row-major [r][n], r <= kLowRankMax;
// `partials` holds kLossPartials * (kLowRankMax + 1) doubles.
constexpr uint32_t kLowRankMax = 16;
hipError_t launch_lowrank_loss(const void *theta, bool bf16, const float *a, const float *U,
                               uint32_t r, uint64_t n, double *partials, double *out,
                               hipStream_t stream);

// Two-layer MLP classifier loss (fp32 parameters, MFMA GEMM, fp64 reduction); with
// `pert` the parameters are read as theta + alpha * z_probe without being written, and with
// `pert` and `out_minus` the loss at theta - alpha * z_probe goes to out_minus as well (the
// workspace then holds both signs' partials).
struct MlpPerturb {
    uint64_t offset;
    uint32_t step, probe;
    float alpha;
    const uint8_t *bits;
};
hipError_t launch_mlp_loss(const float *params, const float *X, const int64_t *labels,
                           uint32_t batch, uint32_t d_in, uint32_t d_hid, uint32_t d_out,
                           double *partial, double *out, const MlpPerturb *pert, Key key,
                           hipStream_t stream, double *out_minus = nullptr);

// Both losses of probes pert.probe .. pert.probe + nprobes - 1 (out_plus[i], out_minus[i]),
// up to kMlpProbesPerLaunch probes per launch sequence, kMlpProbesPerWave of them per wave
// sharing every operand load (ZO_MLP_PROBES_PER_WAVE overrides: 1, 2, 4, 8; 4 at most on 32-wide tiles); pert.bits (if
// given) holds nprobes packed rows.  With out_clean the first launch sequence also computes
// the loss at the unperturbed parameters (bit-equal to launch_mlp_loss without pert).  The
// workspace holds 2 * min(nprobes, kMlpProbesPerLaunch) + 1 slots of partial logits and row
// losses.
constexpr uint32_t kMlpProbesPerLaunch = 64;
constexpr uint32_t kMlpProbesPerWave = 2;
hipError_t launch_mlp_loss_probes(const float *params, const float *X, const int64_t *labels,
                                  uint32_t batch, uint32_t d_in, uint32_t d_hid, uint32_t d_out,
                                  double *partial, const MlpPerturb &pert, uint32_t nprobes,
                                  Key key, double *out_plus, double *out_minus,
                                  double *out_clean, hipStream_t stream);

// Target of a row that counts for nothing (ZO_IGNORE_TOKEN).
constexpr int64_t kIgnoreToken = -100;
// Most threads that the language-model operators put into one launch (the hardware's limit is
// 2^32 - 1).
constexpr uint64_t kLaunchThreads = (uint64_t)1 << 31;
// Bytes of the last cache (256 MB).  What is read once and does not fit is read past it: the
// loads then run at 6.4 TB/s instead of 5.8.
constexpr uint64_t kLastCache = (uint64_t)256 << 20;
// Most alternatives one zo_token_logprobs call gives.
constexpr uint32_t kMaxTopK = 32;
// Largest rank of an adapter.
constexpr uint32_t kMaxRank = 128;

// Per row of logits [rows][stride]: log probability of its target, entropy, top_k
// alternatives (value descending, index ascending).  targets, entropy may be nullptr.
hipError_t launch_token_logprobs(const void *logits, bool bf16, uint64_t rows, uint32_t vocab,
                                 uint64_t stride, const int64_t *targets, float *logp,
                                 float *entropy, uint32_t top_k, int64_t *top_ids,
                                 float *top_logp, hipStream_t stream);

// loss[g] = -mean of logp over the counted rows of [starts[g], starts[g + 1]).
hipError_t launch_group_loss(const float *logp, const int64_t *targets, const int64_t *starts,
                             uint32_t n_groups, uint64_t rows, double *loss, hipStream_t stream);

// Raise the dynamic-LDS limits of the product kernels on the current device (from zo_init).
hipError_t prepare_products();

// The groups of rows of one zo_adapter_project call (device pointers).
struct AdapterArgs {
    uint64_t rows;
    uint32_t d_in, d_out, rank, n_adapters, n_groups, n_probes;
    float scale;
    const int64_t *starts;
    const int32_t *ids, *probes;   // probes nullptr: no group is moved
    const float *alphas;
    const uint8_t *bits;           // n_probes packed rows over all adapters' parameters
    uint64_t bits_stride;
};
// How a product of rows x features is cut into workgroups: 32 features (or 64) and all of at
// most 32 rows, or 64 rows while that is one workgroup per CU in bf16, three in fp32 (64 rows,
// bf16 7168 to 7168: 39 us in tiles of 64 x 64, 22 so; 5120 to 20480 44 and 48; fp32 2048 to
// 2048 50 and 25); tiles of 64 x 64; tiles of 256 x 256.
enum class Shape { few, mid, big };
// Tiles of 256 x 256 that run at once (one per CU), the most slices of one along k, the fewest
// steps of 128 bytes of k that make a slice, and the workspace of all slices of a call.
constexpr uint32_t kBigSlots = 256, kBigSlices = 16, kBigSliceSteps = 4;
constexpr uint64_t kBigSliceBytes = (uint64_t)kBigSlots * 256 * 256 * 4;
// Slices of each of `over` tiles that do not fill a round.
__host__ __device__ constexpr uint32_t big_slices(uint32_t over, uint32_t steps)
{
    uint32_t s = over ? kBigSlots / over : 1;
    s = s > kBigSlices ? kBigSlices : s;
    return s > steps / kBigSliceSteps ? steps / kBigSliceSteps : s;
}
// The shape by estimated time.  Measured per step of 128 bytes of k: a round of 256 tiles of
// 256 x 256 takes 1.45 us (bf16; fp32 7.5), a round of 512 tiles of 64 x 64 0.48 us (1.17),
// or 0.33 us (0.77) while they are at most one per CU (fp32 128 rows, 4096 to 8192: 106 us; in
// sliced tiles of 256 x 256 165); slices cost 25 us to write and add up.
inline Shape product_shape(uint64_t rows, uint32_t features, uint32_t k, bool bf16)
{
    if (rows <= 32 || (rows <= 64 && features <= 32u * 256 * (bf16 ? 1 : 3))) return Shape::few;
    const auto tiles = [&](uint64_t size) {
        return ((uint64_t)features + size - 1) / size * ((rows + size - 1) / size);
    };
    const uint32_t steps = (k + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32);
    const uint64_t m = tiles(64), b = tiles(256), over = b % kBigSlots;
    const double mid = m <= 256 ? (bf16 ? 0.33 : 0.77) : (bf16 ? 0.48 : 1.17) * ((m + 511) / 512);
    const uint32_t slices = big_slices((uint32_t)over, steps);
    const double part = over == 0 ? 0.0 : slices > 1 ? 1.0 / slices : 1.0;
    const double big = (bf16 ? 1.45 : 7.5) * ((double)(b / kBigSlots) + part);
    return steps * big + (over && slices > 1 ? 25.0 : 0.0) <= steps * mid ? Shape::big : Shape::mid;
}
// Features of a workgroup of Shape::few.  With more than 16 rows a CU holds one, and a round of
// 64 features takes 1.6 times one of 32.
inline uint32_t few_features(uint64_t rows, uint32_t features)
{
    const auto rounds = [&](uint32_t each) { return ((features - 1) / each + 256) / 256; };
    return rows > 16 && rows <= 32 && 1.6 * rounds(64) <= rounds(32) ? 64 : 32;
}
// Features of one partial softmax: a wave's.
inline uint32_t shape_part(Shape s, uint64_t rows, uint32_t features)
{
    return s == Shape::big ? 128 : s == Shape::mid ? 32 : few_features(rows, features);
}
// The most of `rows` rows or fewer that take a shape that is big, or one that is not; 0: none do.
// A caller keeps one workspace for its largest batch, and a smaller one may need more for its
// shape, so that sizes look at all counts.  From 64 rows on a shape lasts to the next multiple of
// 64; up to 32 rows it is few.
inline uint64_t most_rows(bool big, uint64_t rows, uint32_t features, uint32_t k, bool bf16)
{
    for (uint64_t r = rows; r > 0; r = r > 64 ? (r - 1) / 64 * 64 : r > 32 ? 32 : 0)
        if ((product_shape(r, features, k, bf16) == Shape::big) == big) return r;
    return 0;
}
// Whether a workspace for up to `rows` rows holds slices, of either type; beyond kShapeRows
// always, so that the search stays short.
constexpr uint64_t kShapeRows = 4096;
inline bool slices_up_to(uint64_t rows, uint32_t features, uint32_t k)
{
    return rows > kShapeRows || most_rows(true, rows, features, k, true) ||
           most_rows(true, rows, features, k, false);
}
// Bytes of x A^T, [rows][rank] floats, and of each row's group.
inline uint64_t adapter_u_bytes(uint64_t rows, uint32_t rank)
{
    return (rows * rank * 4 + rows * 4 + 255) / 256 * 256;
}
// u: adapter_u_bytes of workspace; slices: kBigSliceBytes if the shape is big, else nullptr.
hipError_t launch_adapter_project(const AdapterArgs &a, bool bf16, const void *x, uint64_t x_stride,
                                  const void *w, const void *bias, const void *adapters, float *u,
                                  float *slices, void *y, uint64_t y_stride, hipStream_t stream);

struct HeadArgs {
    uint64_t rows, x_stride;
    uint32_t k, features;
    const int64_t *targets;        // nullptr: entropies of all rows
    float *logp, *entropy;
    void *workspace;
};
// Rows whose partial statistics are held at once.
constexpr uint64_t kHeadPlaces = 16384;
struct HeadSpace {
    uint32_t *count, *list;
    float *m, *s, *t, *tl, *slices;
    Shape shape;
    uint32_t parts;            // partial statistics of a row
    uint64_t bytes;
};
inline HeadSpace head_space(uint64_t rows, uint32_t k, uint32_t features, bool bf16, void *base)
{
    const uint64_t places = rows < kHeadPlaces ? rows : kHeadPlaces;
    HeadSpace s;
    s.shape = product_shape(places, features, k, bf16);
    const uint32_t part = shape_part(s.shape, places, features);
    s.parts = (features + part - 1) / part;
    // the most partial statistics of this and of all smaller counts
    const auto partial = [&](uint64_t n, uint64_t each) { return (features + each - 1) / each * n; };
    const uint64_t other = partial(most_rows(false, places, features, k, bf16), 32);
    const uint64_t big = partial(places, 128), most = big > other ? big : other;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        void *p = base ? static_cast<char *>(base) + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    s.count = static_cast<uint32_t *>(take(4));
    s.list = static_cast<uint32_t *>(take(rows * 4));
    s.m = static_cast<float *>(take(most * 4));
    s.s = static_cast<float *>(take(most * 4));
    s.t = static_cast<float *>(take(most * 4));
    s.tl = static_cast<float *>(take(places * 4));
    s.slices = nullptr;
    if (slices_up_to(places, features, k)) {
        float *slices = static_cast<float *>(take(kBigSliceBytes));
        if (s.shape == Shape::big) s.slices = slices;
    }
    s.bytes = at;
    return s;
}
hipError_t launch_head_logprobs(const HeadArgs &h, bool bf16, const void *x, const void *w,
                                hipStream_t stream);

// Diagnostic: every 16-byte word of buf (bytes % 16 == 0) <- word ^ mask, in place;
// slice_bytes > 0 (a multiple of 8 KiB) issues it as one launch per slice of that size.
hipError_t launch_stream_rmw(void *buf, uint64_t bytes, uint32_t mask, int num_cus,
                             hipStream_t stream, uint64_t slice_bytes = 0);

}  // namespace zo
