// batch.cu - entry points of the batch operators (moe_group_route, moe_grouped_matmul,
// moe_grouped_wgrad, moe_verify_draft): argument checks, then one launcher each.
#include "../../include/moe.h"
#include "group_route.h"
#include "grouped.h"
#include "verify.h"

#include <unistd.h>

#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

namespace {

// What a device needs once: kernel attributes, its SM count, and the host-visible word that a kernel whose wait ran
// out sets.  Made by the first call on the device, kept for the life of the process.
struct Device {
  int num_sms;
  uint32_t* status;                 // as the device sees it
  volatile uint32_t* host_status;
  std::atomic<unsigned long long> wait_cycles;   // bound of the kernels' waits

  moe::WaitLimit wait() const { return {status, wait_cycles.load(std::memory_order_relaxed)}; }
};
constexpr unsigned long long kWaitCycles = 2000000000ull;   // about a second
constexpr int kMaxDevices = 64;
std::mutex g_mu;
std::atomic<Device*> g_device[kMaxDevices];

moe_status device_setup(int dev, Device** out) {
  std::lock_guard<std::mutex> lk(g_mu);
  if ((*out = g_device[dev].load())) return MOE_OK;
  int num_sms = 0;
  if (cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      moe::grouped_any_set_attributes() != cudaSuccess || moe::grouped_pair_set_attributes() != cudaSuccess ||
      moe::grouped_few_set_attributes() != cudaSuccess || moe::verify_set_attributes() != cudaSuccess ||
      moe::group_route_set_attributes() != cudaSuccess) {
    cudaGetLastError();
    return MOE_ECUDA;
  }
  // the word stands in a page of its own, registered
  const size_t page = (size_t)sysconf(_SC_PAGESIZE);
  void* word = nullptr;
  *out = new (std::nothrow) Device{num_sms, nullptr, nullptr, {kWaitCycles}};
  if (!*out || posix_memalign(&word, page, page) != 0) {
    delete *out;
    return MOE_ENOMEM;
  }
  memset(word, 0, page);
  void* on_device = nullptr;
  if (cudaHostRegister(word, page, cudaHostRegisterMapped | cudaHostRegisterPortable) != cudaSuccess ||
      cudaHostGetDevicePointer(&on_device, word, 0) != cudaSuccess) {
    cudaGetLastError();
    free(word);
    delete *out;
    return MOE_ECUDA;
  }
  (*out)->host_status = static_cast<volatile uint32_t*>(word);
  (*out)->status = static_cast<uint32_t*>(on_device);
  g_device[dev].store(*out);
  return MOE_OK;
}

// the current device, set up; MOE_ETIMEOUT once a wait ran out there
moe_status current_device(Device** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return MOE_ECUDA;
  }
  *out = g_device[dev].load(std::memory_order_acquire);
  if (!*out) {
    const moe_status st = device_setup(dev, out);
    if (st != MOE_OK) return st;
  }
  return *(*out)->host_status ? MOE_ETIMEOUT : MOE_OK;
}

bool is_dtype(int t, bool fp32) { return t == MOE_T_BF16 || t == MOE_T_FP16 || (fp32 && t == MOE_T_FP32); }
size_t dtype_bytes(int t) { return t == MOE_T_FP32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// rows of `len` elements `ld` apart that do not overlap, all of them within 2^62 bytes
bool rows_fit(long long rows, long long ld, long long len) {
  return rows >= 0 && ld >= len && ld < (1ll << 40) && (rows == 0 || ld <= (1ll << 60) / rows);
}

// `rows` rows of `len` elements in each of B sequences, none on another: one sequence behind the other, or the sequences' first
// rows, then their second ones, and so on
bool sequences_fit(int B, long long seq, int rows, long long row, int len) {
  if (!rows_fit(rows, row, len)) return false;
  return B == 1 || rows_fit(B, seq, (rows - 1) * row + len) || (rows_fit(B, seq, len) && rows_fit(rows, row, (B - 1) * seq + len));
}

moe_status done(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ECUDA;
}

constexpr long long kMaxRows = 1ll << 30;
constexpr int kMaxDim = 1 << 24;

bool product_ok(int groups, long long m, int n, int k, int dtype, int out_dtype) {
  return groups >= 1 && groups <= 1024 && m >= 0 && m <= kMaxRows && n >= 1 && n <= kMaxDim && k >= 1 && k <= kMaxDim &&
         is_dtype(dtype, false) && is_dtype(out_dtype, true);
}

// Whether the kernel for few rows a group takes a forward product, by the mean over the groups that m rows can reach, as
// the groups' sizes are not known here: tiles of nt rows, four times the mean, so that uneven groups fit too.  Measured
// (DeepSeek-V3- and Mixtral-shaped layers, us for nt 16 / 32 / 64 / the pair kernel): mean 1: 73 / 73 / 75 / 79; mean 8:
// 2102 / 2076 / 2096 / 2189; mean 16: 390 / 284 / 275 / 281; mean 24: 499 / 319 / 278 / 282; mean 32: 622 / 417 / 308 / 284.  Uneven groups at mean 16 (64 experts, n =
// 4096, k = 14336): half of the rows in one group 1118 and 1125 us by the pair kernel, all of them in four groups 153 and 91, in one
// 145 and 72; 256 experts 539 and 275: an expert's weights are then read by more tiles than the pair kernel makes.
int few_rows_tile(long long m, int groups) {
  const long long reach = m < groups ? m : groups;
  return m < 1 ? 0 : m <= 4 * reach ? 16 : m <= 8 * reach ? 32 : m <= 16 * reach ? 64 : 0;
}
// And the blocks that share a tile's k: as many as bring 1.5 blocks an SM from the tiles that m rows spread evenly make,
// 512 elements each at least.  Measured (down product, k = 14336, 64 tiles, cluster 1 / 2 / 4 / 8): 57 / 42 / 39 / 42 us;
// 450 tiles of k = 2048: 40 / 45 / 53 / 82 us.  Tiles full of rows gain less: one block an SM (192 tiles, k = 2048: 13 / 18 us).
// It also takes products of which the pair kernel would keep a third of its pairs busy or fewer (4096 rows in 4 groups, n =
// 128: k = 512 14 and 9 us, k = 4096 34 and 21 us; n = 512, k = 4096 36 and 71 us), or whose tiles of 32 rows stand on the SMs
// all at once, taken as the most that m rows make, while k is not long (pair kernel and this one: 768 rows in 32 groups, n = 512,
// k = 512 7.3 and 7.1 us; in 8 groups, k = 2048 13.2 and 10.4, n = 768 13.2 and 13.4, 192 tiles), and up to half of the pairs where a tile of 64 rows covers a group
// and k is long enough to share out (308 rows in 7 groups, n = 928, k = 14280: 57 and 39 us; n = 1024, k = 1024: 9.2 and 10.4;
// at n = 2048, k = 4096, 64 tiles, 26 and 27).
bool few_rows(const moe::GroupedProblem& p, int num_sms, int* nt, int* cluster) {
  *nt = few_rows_tile(p.m, p.groups);
  const int n_out = p.swiglu ? p.n / 2 : p.n, width = p.swiglu ? 128 : 256;
  const long long pair_tiles = (p.m / 256 + (p.m < p.groups ? p.m : p.groups)) * ((n_out + width - 1) / width);
  const double reached = p.groups * (1 - std::pow(1 - 1.0 / p.groups, (double)p.m));
  auto tiles_of = [&](int rows) { return (reached + p.m / rows) * std::ceil(n_out / (width / 2.0)); };
  if (!*nt && (pair_tiles <= num_sms / 6 || (p.k <= 2048 && tiles_of(32) <= 2 * num_sms))) *nt = 32;
  if (!*nt && pair_tiles <= num_sms / 4 && p.k >= 4096 && p.m <= 48ll * p.groups) *nt = 64;
  if (!*nt) return false;
  const double tiles = tiles_of(*nt);
  *cluster = 1;
  const double most = (few_rows_tile(p.m, p.groups) ? 1.5 : 1.0) * num_sms;
  while (*cluster < 8 && tiles * *cluster < most && p.k / (2 * *cluster) >= 512) *cluster *= 2;
  return true;
}

size_t row_copy_bytes(long long m, int len) { return (size_t)m * ((len + 7) / 8 * 8) * 2; }

// Where an operand's rows are named by number: copies them into ws (m rows), and makes the operand the copy.
struct Operand {
  const uint16_t** base;
  const int** rows;
  long long *nrows, *ld;
  int len;
};
cudaError_t copy_operand(const Operand& o, const moe::GroupedProblem& p, uint16_t* ws, int num_sms, cudaStream_t s) {
  const int ld = (o.len + 7) / 8 * 8;
  const moe::RowCopy c{*o.base, ws, *o.rows, p.offsets, *o.nrows, *o.ld, p.m, p.groups, o.len, ld};
  *o.base = ws;
  *o.rows = nullptr;
  *o.nrows = p.m;
  *o.ld = ld;
  return moe::launch_copy_rows(c, num_sms, s);
}

// The kernel of a product.  TMA wants 16-byte aligned addresses and strides, and many rows side by side, so those named by
// number are copied into the workspace first.
struct Plan {
  int kernel;              // moe_grouped_kernel_id
  int nt, cluster;         // of the few-rows kernel
  size_t need_a, need_b;   // bytes of the copies that the pair kernel takes
};
Plan plan_product(const moe::GroupedProblem& p, bool wgrad, int num_sms, size_t workspace_bytes) {
  Plan pl{MOE_GROUPED_ANY, 0, 0, p.a_rows ? row_copy_bytes(p.m, wgrad ? p.n : p.k) : 0, p.b_rows ? row_copy_bytes(p.m, p.k) : 0};
  if (!wgrad && few_rows(p, num_sms, &pl.nt, &pl.cluster) && moe::grouped_maps(p, false, true, nullptr))
    pl.kernel = MOE_GROUPED_FEW;
  // (the copies lie no worse than the operands)
  else if (p.m > 0 && workspace_bytes >= pl.need_a + pl.need_b && moe::grouped_maps(p, wgrad, false, nullptr))
    pl.kernel = MOE_GROUPED_PAIR;
  return pl;
}

moe_status run_product(moe::GroupedProblem p, bool wgrad, void* workspace, size_t workspace_bytes, cudaStream_t s) {
  Device* d;
  const moe_status st = current_device(&d);
  if (st != MOE_OK) return st;
  const Operand a{&p.a, &p.a_rows, &p.a_nrows, &p.lda, wgrad ? p.n : p.k};
  const Operand b{&p.b, &p.b_rows, &p.b_nrows, &p.ldb, p.k};
  const Plan pl = plan_product(p, wgrad, d->num_sms, workspace_bytes);
  cudaError_t e = cudaSuccess;
  if (pl.kernel == MOE_GROUPED_FEW && moe::launch_grouped_few(p, pl.nt, pl.cluster, d->wait(), s, &e)) return done(e);
  if (pl.kernel == MOE_GROUPED_PAIR) {
    uint16_t* ws = static_cast<uint16_t*>(workspace);
    if (pl.need_a) e = copy_operand(a, p, ws, d->num_sms, s);
    if (pl.need_b && e == cudaSuccess) e = copy_operand(b, p, ws + pl.need_a / 2, d->num_sms, s);
    if (e != cudaSuccess) return done(e);
    if (moe::launch_grouped_pair(p, wgrad, d->num_sms, d->wait(), s, &e)) return done(e);
  }
  return done(moe::launch_grouped_any(p, wgrad, d->wait(), s));
}

}  // namespace

extern "C" size_t moe_group_route_workspace(int T, int E, int k) {
  if (T < 1 || E < 1 || E > 1024 || k < 1 || k > E || k > 32 || (long long)T * k > 0x7fffffffLL) return 0;
  return moe::group_route_plan(T, E, k).workspace;
}

extern "C" moe_status moe_group_route(const void* logits, long long ld, int dtype, int T, int E, int k, int router,
                                      int* idx, float* weights, int* offsets, int* rows, int* pairs, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!logits || !idx || !weights || !offsets || !rows || !pairs) return MOE_EINVAL;
  if (!is_dtype(dtype, true) || T < 1 || E < 1 || E > 1024 || k < 1 || k > E || k > 32) return MOE_EINVAL;
  if ((long long)T * k > 0x7fffffffLL || !rows_fit(T, ld, E)) return MOE_EINVAL;
  if (router != MOE_ROUTER_SOFTMAX_TOPK_RENORM && router != MOE_ROUTER_SIGMOID_TOPK_NORM) return MOE_EINVAL;
  if (!aligned(logits, dtype_bytes(dtype)) || !aligned(idx, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
      !aligned(rows, 4) || !aligned(pairs, 4) || !aligned(workspace, 16))
    return MOE_EINVAL;
  const moe::GroupRoutePlan plan = moe::group_route_plan(T, E, k);
  if (plan.workspace && (!workspace || workspace_bytes < plan.workspace)) return MOE_EINVAL;
  moe::GroupRouteArgs a{logits, ld, dtype, T, E, k, router, idx, weights, offsets, rows, pairs,
                        static_cast<int*>(workspace), plan.blocks, plan.per_block};
  Device* d;
  const moe_status st = current_device(&d);
  if (st != MOE_OK) return st;
  return done(moe::launch_group_route(a, (cudaStream_t)stream));
}

extern "C" size_t moe_grouped_workspace(long long m, int k, int groups) {
  if (m < 0 || m > kMaxRows || k < 1 || k > kMaxDim || groups < 1 || groups > 1024) return 0;
  return few_rows_tile(m, groups) ? 0 : row_copy_bytes(m, k);
}

extern "C" size_t moe_grouped_wgrad_workspace(long long m, int len) {
  return m < 0 || m > kMaxRows || len < 1 || len > kMaxDim ? 0 : row_copy_bytes(m, len);
}

namespace {

// the arguments checked, and as the kernels take them
moe_status matmul_problem(const moe_grouped_args* a, moe::GroupedProblem* out) {
  if (!a || (!a->x && a->x_rows != 0) || !a->w || !a->offsets || !a->out) return MOE_EINVAL;
  if (!product_ok(a->groups, a->m, a->n, a->k, a->dtype, a->out_dtype)) return MOE_EINVAL;
  if (a->layout != MOE_GROUP_NK && a->layout != MOE_GROUP_KN) return MOE_EINVAL;
  if (a->act != MOE_ACT_NONE && a->act != MOE_ACT_SWIGLU) return MOE_EINVAL;
  const bool sw = a->act == MOE_ACT_SWIGLU, kn = a->layout == MOE_GROUP_KN;
  if (sw && (kn || a->n % 2)) return MOE_EINVAL;
  if (!rows_fit(a->x_rows, a->ldx, a->k) || !rows_fit(kn ? a->k : a->n, a->ldw, kn ? a->n : a->k) ||
      !rows_fit(a->out_rows_n, a->ldo, sw ? a->n / 2 : a->n) || a->w_stride < 0 || a->w_stride >= (1ll << 50))
    return MOE_EINVAL;
  if ((!a->rows && a->m > a->x_rows) || (!a->out_rows && a->m > a->out_rows_n)) return MOE_EINVAL;
  if (!aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->out, dtype_bytes(a->out_dtype)) || !aligned(a->offsets, 4) ||
      !aligned(a->rows, 4) || !aligned(a->out_rows, 4) || !aligned(a->workspace, 16) ||
      (!a->workspace && a->workspace_bytes))
    return MOE_EINVAL;
  moe::GroupedProblem& p = *out;
  p = {};
  p.a = static_cast<const uint16_t*>(a->x);
  p.b = static_cast<const uint16_t*>(a->w);
  p.d = a->out;
  p.offsets = a->offsets;
  p.a_rows = a->rows;
  p.d_rows = a->out_rows;
  p.a_nrows = a->x_rows;
  p.lda = a->ldx;
  p.ldb = a->ldw;
  p.b_stride = a->w_stride;
  p.d_nrows = a->out_rows_n;
  p.ldd = a->ldo;
  p.m = a->m;
  p.groups = a->groups;
  p.n = a->n;
  p.k = a->k;
  p.dtype = a->dtype;
  p.out_dtype = a->out_dtype;
  p.kn = kn;
  p.swiglu = sw;
  return MOE_OK;
}

moe_status wgrad_problem(const moe_grouped_wgrad_args* a, moe::GroupedProblem* out) {
  if (!a || !a->offsets || !a->dw) return MOE_EINVAL;
  if (a->m != 0 && ((!a->dy && a->dy_rows_n != 0) || (!a->x && a->x_rows_n != 0))) return MOE_EINVAL;
  if (!product_ok(a->groups, a->m, a->n, a->k, a->dtype, a->out_dtype)) return MOE_EINVAL;
  if (!rows_fit(a->dy_rows_n, a->lddy, a->n) || !rows_fit(a->x_rows_n, a->ldx, a->k) || !rows_fit(a->n, a->lddw, a->k) ||
      a->dw_stride < (a->n - 1) * a->lddw + a->k || a->dw_stride >= (1ll << 50))
    return MOE_EINVAL;
  if ((!a->dy_rows && a->m > a->dy_rows_n) || (!a->x_rows && a->m > a->x_rows_n)) return MOE_EINVAL;
  if (!aligned(a->dy, 2) || !aligned(a->x, 2) || !aligned(a->dw, dtype_bytes(a->out_dtype)) || !aligned(a->offsets, 4) ||
      !aligned(a->dy_rows, 4) || !aligned(a->x_rows, 4) || !aligned(a->workspace, 16) ||
      (!a->workspace && a->workspace_bytes))
    return MOE_EINVAL;
  moe::GroupedProblem& p = *out;
  p = {};
  p.a = static_cast<const uint16_t*>(a->dy);
  p.b = static_cast<const uint16_t*>(a->x);
  p.d = a->dw;
  p.offsets = a->offsets;
  p.a_rows = a->dy_rows;
  p.b_rows = a->x_rows;
  p.a_nrows = a->dy_rows_n;
  p.lda = a->lddy;
  p.b_nrows = a->x_rows_n;
  p.ldb = a->ldx;
  p.ldd = a->lddw;
  p.d_stride = a->dw_stride;
  p.m = a->m;
  p.groups = a->groups;
  p.n = a->n;
  p.k = a->k;
  p.dtype = a->dtype;
  p.out_dtype = a->out_dtype;
  return MOE_OK;
}

}  // namespace

extern "C" moe_status moe_grouped_matmul(const moe_grouped_args* a, void* stream) {
  moe::GroupedProblem p;
  const moe_status st = matmul_problem(a, &p);
  if (st != MOE_OK || p.m == 0) return st;
  return run_product(p, false, a->workspace, a->workspace_bytes, (cudaStream_t)stream);
}

extern "C" moe_status moe_grouped_wgrad(const moe_grouped_wgrad_args* a, void* stream) {
  moe::GroupedProblem p;
  const moe_status st = wgrad_problem(a, &p);
  if (st != MOE_OK) return st;
  return run_product(p, true, a->workspace, a->workspace_bytes, (cudaStream_t)stream);
}

extern "C" moe_status moe_debug_batch_wait(long long cycles) {
  if (cycles > 1ll << 36) return MOE_EINVAL;
  Device* d;
  const moe_status st = current_device(&d);
  if (st != MOE_OK && st != MOE_ETIMEOUT) return st;
  d->wait_cycles.store(cycles < 0 ? kWaitCycles : (unsigned long long)cycles);
  *d->host_status = 0;
  return MOE_OK;
}

extern "C" int moe_grouped_kernel(const moe_grouped_args* a, int num_sms) {
  moe::GroupedProblem p;
  return matmul_problem(a, &p) != MOE_OK || p.m == 0 || num_sms < 1 ? MOE_GROUPED_NONE
                                                                    : plan_product(p, false, num_sms, a->workspace_bytes).kernel;
}

extern "C" int moe_grouped_wgrad_kernel(const moe_grouped_wgrad_args* a, int num_sms) {
  moe::GroupedProblem p;
  return wgrad_problem(a, &p) != MOE_OK || num_sms < 1 ? MOE_GROUPED_NONE
                                                       : plan_product(p, true, num_sms, a->workspace_bytes).kernel;
}

extern "C" moe_status moe_verify_draft(const moe_verify_args* a, void* stream) {
  if (!a || !a->p || !a->u || !a->accepted || !a->tokens) return MOE_EINVAL;
  if (a->B < 1 || a->D < 0 || a->D > 31 || (a->D && !a->draft) || a->V < 1 || a->V > (1 << 30) || !is_dtype(a->dtype, true))
    return MOE_EINVAL;
  if (!sequences_fit(a->B, a->p_seq, a->D + 1, a->p_row, a->V)) return MOE_EINVAL;
  if (a->q && a->D && !sequences_fit(a->B, a->q_seq, a->D, a->q_row, a->V)) return MOE_EINVAL;
  const size_t el = dtype_bytes(a->dtype);
  if (!aligned(a->p, el) || !aligned(a->q, el) || !aligned(a->draft, 4) || !aligned(a->lengths, 4) || !aligned(a->u, 4) ||
      !aligned(a->accepted, 4) || !aligned(a->tokens, 4))
    return MOE_EINVAL;
  moe::VerifyArgs v{a->p, a->q, a->draft, a->lengths, a->u, a->accepted, a->tokens,
                    a->p_seq, a->p_row, a->q_seq, a->q_row, a->B, a->D, a->V, a->dtype};
  Device* d;
  const moe_status st = current_device(&d);
  if (st != MOE_OK) return st;
  return done(moe::launch_verify(v, d->num_sms, (cudaStream_t)stream));
}
