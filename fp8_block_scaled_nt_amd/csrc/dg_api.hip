// C ABI of the FP8 block-scaled NT GEMM library (declared in include/dg.h):
// argument validation, per-shape choice among the compile-time tile
// configurations, and the kernel launches.  The pages' DeepGEMM compiles a
// kernel per shape at run time ("DeepSeek open-source week day 3",
// technical features, JIT item); here every configuration is compiled ahead
// of time for gfx950 and the host picks one per call from (M, N, K, groups,
// CU count), which keeps the call free of compilation, allocation and
// synchronisation.
#include "../../include/dg.h"

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>
#include <unordered_map>
#include <vector>

#include "gemm_kernel.h"
#include "kv8_kernel.h"
#include "latent_kernel.h"
#include "quant_kernel.h"
#include "skinny_kernel.h"
#include "w4_kernel.h"

namespace {

thread_local std::string g_last_error;
// one-shot profiling events for the next GEMM launch on this thread
thread_local hipEvent_t g_prof_start = nullptr;
thread_local hipEvent_t g_prof_stop = nullptr;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

int ok() {
  g_last_error.clear();
  return DG_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sfa_ld(int m) { return (m + 3) / 4 * 4; }

bool log_enabled() {
  static int v = -1;
  if (v < 0) {
    const char* e = getenv("DG_LOG");
    v = (e && *e && *e != '0') ? 1 : 0;
  }
  return v == 1;
}

// ---- per-device facts, queried once per device
struct DeviceInfo {
  int cus = 0;
  bool ok = false;
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];

int current_device(int* dev, DeviceInfo** info) {
  // hipGetDevice is a thread-local read; it fails when no device is visible
  if (hipGetDevice(dev) != hipSuccess || *dev < 0 || *dev >= kMaxDevices) {
    (void)hipGetLastError();
    return fail(DG_ERR_NO_DEVICE, "no HIP device is visible");
  }
  const int d = *dev;
  std::call_once(g_dev_once[d], [d]() {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, d) != hipSuccess) return;
    g_dev[d].cus = prop.multiProcessorCount;
    g_dev[d].ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  });
  if (!g_dev[d].ok) return fail(DG_ERR_NO_DEVICE, "device %d is not a gfx950 GPU", d);
  *info = &g_dev[d];
  return DG_OK;
}

// ---- tile configurations (compile-time instantiations; the host picks one)
struct Config {
  const char* name;
  int variant, bm, bn, wm, wn, nst, sched, dtype, epi;
  const void* fn;
  int smem;
  int threads() const { return wm * wn * 64; }
};

template <int BM, int BN, int WM, int WN, int NST, int VAR, int SCHED = dg::kInterleaved, int DT = dg::kFp8,
          int EPI = dg::kEpiBf16>
Config make_config(const char* name) {
  return Config{name, VAR, BM, BN, WM, WN, NST, SCHED, DT, EPI,
                reinterpret_cast<const void*>(&dg::gemm_fp8_nt_kernel<BM, BN, WM, WN, NST, VAR, SCHED, DT, EPI>),
                dg::Smem<BM, BN, NST, DT == dg::kFp4 ? 2 : 1, SCHED == dg::kSingleB>::kBytes};
}

const Config* configs(int* count) {
  static const Config table[] = {
      // dense
      make_config<256, 256, 2, 4, 2, dg::kDense>("dense_256x256_w8_s2"),
      make_config<256, 256, 2, 4, 2, dg::kDense, dg::kPingPong>("dense_256x256_w8_s2_pp"),
      make_config<128, 256, 1, 4, 2, dg::kDense, dg::kSingleB>("dense_128x256_w4_s2_sb"),
      make_config<256, 224, 4, 2, 2, dg::kDense>("dense_256x224_w8_s2"),
      make_config<128, 256, 1, 4, 3, dg::kDense>("dense_128x256_w4_s3_wide"),
      make_config<256, 128, 4, 2, 3, dg::kDense>("dense_256x128_w8_s3"),
      make_config<256, 128, 2, 2, 2, dg::kDense>("dense_256x128_w4_s2"),
      make_config<256, 128, 2, 2, 3, dg::kDense>("dense_256x128_w4_s3"),
      make_config<128, 256, 2, 2, 3, dg::kDense>("dense_128x256_w4_s3"),
      make_config<128, 256, 2, 4, 3, dg::kDense>("dense_128x256_w8_s3"),
      make_config<128, 128, 2, 2, 3, dg::kDense>("dense_128x128_w4_s3"),
      make_config<128, 128, 2, 2, 2, dg::kDense>("dense_128x128_w4_s2"),
      make_config<64, 64, 1, 4, 3, dg::kDense>("dense_64x64_w4_s3"),
      // skinny M: split-K over workgroups
      make_config<64, 64, 1, 4, 8, dg::kDense>("dense_64x64_w4_s8"),
      make_config<64, 32, 2, 2, 4, dg::kDense>("dense_64x32_w4_s4"),
      // the same tile consuming two or three slabs per barrier step
      make_config<64, 32, 2, 2, 4, dg::kDense, dg::kPair>("dense_64x32_w4_s4_pair"),
      make_config<64, 32, 2, 2, 6, dg::kDense, dg::kTriple>("dense_64x32_w4_s6_triple"),
      make_config<64, 64, 1, 4, 4, dg::kDense, dg::kPair>("dense_64x64_w4_s4_pair"),
      // contiguous (block rows <= the 128-row alignment)
      make_config<128, 256, 2, 4, 3, dg::kContiguous>("contig_128x256_w8_s3"),
      make_config<128, 128, 2, 2, 3, dg::kContiguous>("contig_128x128_w4_s3"),
      make_config<128, 128, 2, 2, 2, dg::kContiguous>("contig_128x128_w4_s2"),
      make_config<128, 256, 2, 4, 2, dg::kContiguous>("contig_128x256_w8_s2"),
      make_config<128, 256, 1, 4, 3, dg::kContiguous>("contig_128x256_w4_s3"),
      make_config<128, 256, 1, 4, 2, dg::kContiguous, dg::kSingleB>("contig_128x256_w4_s2_sb"),
      make_config<128, 256, 1, 4, 2, dg::kContiguous>("contig_128x256_w4_s2"),
      make_config<64, 64, 1, 4, 3, dg::kContiguous>("contig_64x64_w4_s3"),
      // masked
      make_config<256, 256, 2, 4, 2, dg::kMasked>("masked_256x256_w8_s2"),
      make_config<256, 256, 2, 4, 2, dg::kMasked, dg::kPingPong>("masked_256x256_w8_s2_pp"),
      make_config<256, 128, 4, 2, 2, dg::kMasked>("masked_256x128_w8_s2"),
      make_config<256, 128, 1, 4, 2, dg::kMasked>("masked_256x128_w4_s2"),
      make_config<256, 128, 1, 4, 3, dg::kMasked>("masked_256x128_w4_s3"),
      make_config<64, 64, 1, 4, 3, dg::kMasked>("masked_64x64_w4_s3"),
      make_config<128, 256, 2, 4, 3, dg::kMasked>("masked_128x256_w8_s3"),
      // K-grouped
      make_config<256, 256, 2, 4, 2, dg::kKGrouped>("kgrouped_256x256_w8_s2"),
      make_config<128, 128, 2, 2, 2, dg::kKGrouped>("kgrouped_128x128_w4_s2"),
      make_config<128, 256, 1, 4, 2, dg::kKGrouped, dg::kSingleB>("kgrouped_128x256_w4_s2_sb"),
      // BF16 dense (find_config matches the dtype too, so DG_FORCE_CONFIG
      // names pick among these only for the bf16 entry point)
      make_config<256, 256, 2, 4, 2, dg::kDense, dg::kInterleaved, dg::kBf16>("bf16_256x256_w8_s2"),
      make_config<128, 128, 2, 2, 2, dg::kDense, dg::kInterleaved, dg::kBf16>("bf16_128x128_w4_s2"),
      make_config<64, 32, 2, 2, 4, dg::kDense, dg::kInterleaved, dg::kBf16>("bf16_64x32_w4_s4"),
      make_config<64, 32, 2, 2, 4, dg::kDense, dg::kPair, dg::kBf16>("bf16_64x32_w4_s4_pair"),
      make_config<64, 64, 1, 4, 3, dg::kDense, dg::kInterleaved, dg::kBf16>("bf16_64x64_w4_s3"),
      // FP4 (e2m1) dense (selected the same way by dtype)
      make_config<256, 256, 2, 4, 2, dg::kDense, dg::kInterleaved, dg::kFp4>("fp4_256x256_w8_s2"),
      make_config<128, 128, 2, 2, 2, dg::kDense, dg::kInterleaved, dg::kFp4>("fp4_128x128_w4_s2"),
      make_config<64, 32, 2, 2, 4, dg::kDense, dg::kInterleaved, dg::kFp4>("fp4_64x32_w4_s4"),
      make_config<64, 32, 2, 2, 6, dg::kDense, dg::kTriple, dg::kFp4>("fp4_64x32_w4_s6_triple"),
      make_config<64, 64, 1, 4, 3, dg::kDense, dg::kInterleaved, dg::kFp4>("fp4_64x64_w4_s3"),
      make_config<64, 64, 1, 4, 4, dg::kDense, dg::kPair, dg::kFp4>("fp4_64x64_w4_s4_pair"),
      // MoE FC1 + SwiGLU + FP8 requantisation, masked layout (a 256-column
      // tile = 128 gate + 128 up columns = one 128-wide block of h)
      make_config<256, 256, 2, 4, 2, dg::kMasked, dg::kPingPong, dg::kFp8, dg::kEpiSwigluFp8>("swiglu_256x256_w8_s2_pp"),
      make_config<256, 256, 2, 4, 2, dg::kMasked, dg::kInterleaved, dg::kFp8, dg::kEpiSwigluFp8>("swiglu_256x256_w8_s2"),
      make_config<128, 256, 2, 4, 3, dg::kMasked, dg::kInterleaved, dg::kFp8, dg::kEpiSwigluFp8>("swiglu_128x256_w8_s3"),
      make_config<64, 256, 1, 4, 3, dg::kMasked, dg::kInterleaved, dg::kFp8, dg::kEpiSwigluFp8>("swiglu_64x256_w4_s3"),
      // the same on the contiguous layout (tile rows within the 128-row alignment)
      make_config<128, 256, 1, 4, 2, dg::kContiguous, dg::kSingleB, dg::kFp8, dg::kEpiSwigluFp8>(
          "swiglu_contig_128x256_w4_s2_sb"),
      make_config<128, 256, 2, 4, 3, dg::kContiguous, dg::kInterleaved, dg::kFp8, dg::kEpiSwigluFp8>(
          "swiglu_contig_128x256_w8_s3"),
      make_config<64, 256, 1, 4, 3, dg::kContiguous, dg::kInterleaved, dg::kFp8, dg::kEpiSwigluFp8>(
          "swiglu_contig_64x256_w4_s3"),
  };
  *count = sizeof(table) / sizeof(table[0]);
  return table;
}

const Config* find_config(const char* name, int variant, int dtype = dg::kFp8, int epi = dg::kEpiBf16) {
  int cnt = 0;
  const Config* t = configs(&cnt);
  for (int i = 0; i < cnt; ++i)
    if (t[i].variant == variant && t[i].dtype == dtype && t[i].epi == epi && strcmp(t[i].name, name) == 0)
      return &t[i];
  return nullptr;
}

// ---- skinny-M fp8 configurations (dense calls with m <= 64): stream-K
// runs of (tile, K slab) units, one unit per wave (skinny_kernel.h)
struct SkinnyConfig {
  const char* name;
  int bn, nw, upw;
  bool sa, sb;  // A / B staged through LDS (whole-row loads) or loaded in the MFMA layout
  const void* fn;
  int threads() const { return nw * 64; }
  // per-wave staging of one unit's rows, later the per-wave fp32 accumulators
  int smem() const {
    const int stage = nw * ((sa ? 64 : 0) + (sb ? bn : 0)) * 128;
    const int red = nw * upw * (64 * bn / 256) * 1024;
    return stage > red ? stage : red;
  }
  int units_per_wg() const { return nw * upw; }
};

template <int BN, int NW, int UPW, bool SA, bool SB>
SkinnyConfig make_skinny(const char* name) {
  return SkinnyConfig{name, BN, NW, UPW, SA, SB,
                      reinterpret_cast<const void*>(&dg::gemm_skinny_kernel<BN, NW, UPW, SA, SB>)};
}

const SkinnyConfig* skinny_configs(int* count) {
  static const SkinnyConfig table[] = {
      make_skinny<32, 16, 1, false, false>("skinny_64x32_w16_direct"),
      make_skinny<32, 16, 1, true, false>("skinny_64x32_w16_stagea"),
      make_skinny<32, 8, 2, true, true>("skinny_64x32_w8_u2_stage"),
      make_skinny<32, 8, 2, false, false>("skinny_64x32_w8_u2_direct"),
      make_skinny<32, 12, 1, true, true>("skinny_64x32_w12_stage"),
      make_skinny<16, 16, 1, false, false>("skinny_64x16_w16_direct"),
      make_skinny<64, 8, 1, true, false>("skinny_64x64_w8_stagea"),
  };
  *count = sizeof(table) / sizeof(table[0]);
  return table;
}

const SkinnyConfig* find_skinny(const char* name) {
  int cnt = 0;
  const SkinnyConfig* t = skinny_configs(&cnt);
  for (int i = 0; i < cnt; ++i)
    if (strcmp(t[i].name, name) == 0) return &t[i];
  return nullptr;
}

// the two ways of a product with 4-bit weights, and of an attention call over the 8-bit cache
constexpr const char* kW4RowsName = "w4_rows";
constexpr const char* kW4TileName = "w4_tile";
constexpr const char* kKv8Split = "kv8_split";
constexpr const char* kKv8Prompt = "kv8_prompt";
// rows of a tile of absorbed attention over latents
constexpr const char* kLatentRows[] = {"latent_rows16", "latent_rows32", "latent_rows64"};
// and queries of a workgroup of expanded attention
constexpr const char* kLatentPrompt[] = {"latent_prompt16", "latent_prompt32", "latent_prompt64", "latent_prompt128"};

// DG_FORCE_CONFIG=<name> pins the configuration of the variant it names (for
// tuning sweeps); an unknown name is an error rather than silently ignored.
int forced_name(const char** name) {
  *name = nullptr;
  const char* e = getenv("DG_FORCE_CONFIG");
  if (!e || !*e) return DG_OK;
  int cnt = 0;
  const Config* t = configs(&cnt);
  bool known = false;
  for (int i = 0; i < cnt; ++i) known = known || strcmp(t[i].name, e) == 0;
  known = known || find_skinny(e) != nullptr || strcmp(e, kKv8Split) == 0 || strcmp(e, kKv8Prompt) == 0 ||
          strcmp(e, kW4RowsName) == 0 || strcmp(e, kW4TileName) == 0;
  for (const char* rows : kLatentRows) known = known || strcmp(e, rows) == 0;
  for (const char* rows : kLatentPrompt) known = known || strcmp(e, rows) == 0;
  if (!known) return fail(DG_ERR_INVALID_ARGUMENT, "DG_FORCE_CONFIG names no configuration: %s", e);
  *name = e;
  return DG_OK;
}

int forced_config(int variant, const Config** out, int dtype = dg::kFp8, int epi = dg::kEpiBf16) {
  *out = nullptr;
  const char* name;
  if (int s = forced_name(&name)) return s;
  if (name) *out = find_config(name, variant, dtype, epi);
  return DG_OK;
}

// The same for calls that choose between two ways: the one pinned, or null.
int forced_way(const char* one, const char* other, const char** way) {
  const char* name;
  *way = nullptr;
  if (int s = forced_name(&name)) return s;
  if (name && strcmp(name, one) == 0) *way = one;
  if (name && strcmp(name, other) == 0) *way = other;
  return DG_OK;
}

std::once_flag g_attr_once;
hipError_t g_attr_err = hipSuccess;
constexpr int kMaxConfigs = 64;
int g_per_cu[kMaxConfigs];  // resident workgroups per CU of each configuration (0: not known)

void set_kernel_attributes() {
  int scnt = 0;
  const SkinnyConfig* st = skinny_configs(&scnt);
  for (int i = 0; i < scnt; ++i) {
    hipError_t e = hipFuncSetAttribute(st[i].fn, hipFuncAttributeMaxDynamicSharedMemorySize, st[i].smem());
    if (e != hipSuccess) g_attr_err = e;
  }
  int cnt = 0;
  const Config* t = configs(&cnt);
  for (int i = 0; i < cnt; ++i) {
    hipError_t e = hipFuncSetAttribute(t[i].fn, hipFuncAttributeMaxDynamicSharedMemorySize, t[i].smem);
    if (e != hipSuccess) {
      g_attr_err = e;
      continue;
    }
    int blocks = 0;
    if (i < kMaxConfigs &&
        hipOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, t[i].fn, t[i].threads(), t[i].smem) == hipSuccess)
      g_per_cu[i] = blocks;
    else
      (void)hipGetLastError();
  }
}

int ensure_kernel_attributes() {
  std::call_once(g_attr_once, set_kernel_attributes);
  if (g_attr_err != hipSuccess)
    return fail(DG_ERR_HIP, "hipFuncSetAttribute: %s", hipGetErrorString(g_attr_err));
  return DG_OK;
}

// Workgroups of configuration c that one CU holds at once (LDS, registers and
// waves permitting); 1 when the runtime could not say.
int per_cu(const Config* c) {
  int cnt = 0;
  const Config* t = configs(&cnt);
  const long i = c - t;
  return (i >= 0 && i < kMaxConfigs && g_per_cu[i] > 0) ? g_per_cu[i] : 1;
}

// ---- split-K workspace: library-owned device memory, one block per
// (device, stream).  Calls on one stream run in stream order, so they can
// share a block; calls on different streams get different blocks and never
// share an arrival counter or a partial tile.  Layout of a block:
// kCounterInts arrival counters (reset by the kernels after use), then the
// partial tiles; the whole block is zeroed when it is made.
//
// A block only grows: the larger block replaces it for later calls on that
// stream, and the old one is retired, never freed, because a launch still in
// flight or a captured graph may use it.  Growing costs a hipMalloc and a
// zero-fill kernel on the calling stream (stream-ordered: no device-wide
// synchronisation).  A call that would grow the block while its stream is
// capturing a graph returns DG_ERR_WORKSPACE instead (dg_reserve_workspace
// sizes the block beforehand).
constexpr size_t kCounterInts = 1 << 16;
struct StreamWorkspace {
  char* base = nullptr;
  size_t bytes = 0;
};
struct DeviceWorkspaces {
  std::mutex mu;
  std::unordered_map<hipStream_t, StreamWorkspace> by_stream;
  std::vector<void*> retired;  // kept until the process ends
};
DeviceWorkspaces g_ws[kMaxDevices];

__global__ void zero_ints_kernel(int* p, long long n) {
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
    p[i] = 0;
}

constexpr size_t kWsHeader = kCounterInts * sizeof(int);  // the counters

int ensure_workspace(int dev, hipStream_t stream, size_t partial_bytes, char** base) {
  DeviceWorkspaces& w = g_ws[dev];
  std::lock_guard<std::mutex> lock(w.mu);
  StreamWorkspace& ws = w.by_stream[stream];
  const size_t need = kWsHeader + partial_bytes;
  if (ws.bytes < need) {
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(stream, &cap);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return fail(DG_ERR_WORKSPACE, "the split-K workspace of this stream must grow to %zu bytes, and the stream's "
                  "capture state cannot be queried (%s)", need, hipGetErrorString(e));
    }
    if (cap != hipStreamCaptureStatusNone)
      return fail(DG_ERR_WORKSPACE, "the split-K workspace of this stream must grow to %zu bytes (it has %zu) while "
                  "the stream is capturing; reserve it first with dg_reserve_workspace", need, ws.bytes);
    size_t alloc = 2 * ws.bytes;
    if (alloc < need) alloc = need;
    if (alloc < ((size_t)4 << 20)) alloc = (size_t)4 << 20;
    void* ptr = nullptr;
    e = hipMalloc(&ptr, alloc);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return fail(DG_ERR_HIP, "hipMalloc(workspace %zu): %s", alloc, hipGetErrorString(e));
    }
    const long long words = (long long)(alloc / sizeof(int));
    hipLaunchKernelGGL(zero_ints_kernel, dim3(1024), dim3(256), 0, stream, (int*)ptr, words);
    e = hipGetLastError();
    if (e != hipSuccess) {
      w.retired.push_back(ptr);
      return fail(DG_ERR_HIP, "workspace zero-fill launch failed: %s", hipGetErrorString(e));
    }
    if (ws.base) w.retired.push_back(ws.base);
    ws.base = (char*)ptr;
    ws.bytes = alloc;
  }
  *base = ws.base;
  return DG_OK;
}

// ---- allocation-free split-K scratch (dg_fp8_gemm_nt_noalloc): one static
// device array, held by every GPU the library runs on until the process
// ends.  Host code never passes the array's name to a kernel (in host code it
// names a host-side stand-in); it uses the device address that
// hipGetSymbolAddress returns, taken once per device with that device current.
constexpr size_t kScratchCounterInts = (size_t)1 << 14;       // arrival counters: tiles per call
constexpr size_t kScratchPartialBytes = (size_t)16 << 20;     // partial tiles
constexpr size_t kScratchHeader = kScratchCounterInts * sizeof(int);
constexpr size_t kScratchBytes = kScratchHeader + kScratchPartialBytes;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

char* g_scratch_ptr[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];
std::once_flag g_scratch_once[kMaxDevices];

int scratch_address(int dev, char** ptr) {
  std::call_once(g_scratch_once[dev], [dev]() {
    void* p = nullptr;
    g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (g_scratch_err[dev] != hipSuccess) (void)hipGetLastError();
    g_scratch_ptr[dev] = (char*)p;
  });
  if (g_scratch_err[dev] != hipSuccess || !g_scratch_ptr[dev])
    return fail(DG_ERR_HIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(g_scratch_err[dev]));
  *ptr = g_scratch_ptr[dev];
  return DG_OK;
}

// Where a split-K call takes its workspace: the calling stream's block, grown
// on demand (fixed == nullptr), or the static scratch of the allocation-free
// entry point (fixed = its device address), whose counters are cleared for
// every call by a fill kernel on the call's stream (a kernel, not a memset,
// so that a captured call records a kernel node).
struct WsSource {
  char* fixed = nullptr;
};

struct WsView {
  int* counters = nullptr;
  char* partial = nullptr;
};

int get_workspace(const WsSource& src, int dev, hipStream_t stream, size_t partial_bytes, long long counters_used,
                  WsView* v) {
  if (!src.fixed) {
    char* base = nullptr;
    if (int s = ensure_workspace(dev, stream, partial_bytes, &base)) return s;
    v->counters = (int*)base;
    v->partial = base + kWsHeader;
    return DG_OK;
  }
  if (partial_bytes > kScratchPartialBytes || counters_used > (long long)kScratchCounterInts)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "this call needs %zu bytes of split-K scratch and %lld counters; the static "
                "scratch holds %zu bytes and %zu counters", partial_bytes, counters_used, kScratchPartialBytes,
                kScratchCounterInts);
  v->counters = (int*)src.fixed;
  v->partial = src.fixed + kScratchHeader;
  hipLaunchKernelGGL(zero_ints_kernel, dim3((unsigned)((counters_used + 255) / 256)), dim3(256), 0, stream,
                     v->counters, counters_used);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DG_ERR_HIP, "scratch counter clear failed: %s", hipGetErrorString(e));
  return DG_OK;
}

// A GEMM's launch: records the events of dg_profile_next_launch if there are any.
hipError_t launch_gemm_kernel(const void* fn, dim3 grid, int threads, void** args, int smem, hipStream_t stream) {
  if (!g_prof_start && !g_prof_stop) return hipLaunchKernel(fn, grid, dim3(threads), args, smem, stream);
  const hipError_t e = hipExtLaunchKernel(fn, grid, dim3(threads), args, smem, stream, g_prof_start, g_prof_stop, 0);
  g_prof_start = g_prof_stop = nullptr;
  return e;
}

int launch(const Config& c, dg::GemmParams& p, int grid, hipStream_t stream) {
  if (int s = ensure_kernel_attributes()) return s;
  if (log_enabled())
    fprintf(stderr, "[dg] %s m=%d n=%d k=%d groups=%d grid=%d threads=%d smem=%d per_cu=%d splits=%d\n", c.name,
            p.m, p.n, p.k, p.num_groups, grid, c.threads(), c.smem, per_cu(&c), p.splits);
  if (grid <= 0) return ok();
  void* args[] = {&p};
  const hipError_t e = launch_gemm_kernel(c.fn, dim3(grid), c.threads(), args, c.smem, stream);
  if (e != hipSuccess) return fail(DG_ERR_HIP, "launch of %s failed: %s", c.name, hipGetErrorString(e));
  return ok();
}

void fill_common(dg::GemmParams& p, const Config& c, int m, int n, int k) {
  p.m = m;
  p.n = n;
  p.k = k;
  p.kb_count = k / 128;
  p.sk_count = p.kb_count;
  p.nb_count = (n + 127) / 128;
  p.sfa_ld = sfa_ld(m);
  p.tiles_m = (m + c.bm - 1) / c.bm;
  p.tiles_n = (n + c.bn - 1) / c.bn;
  // With one row of tiles (per group) no two tiles read the same B bytes, so
  // B streams through with the non-temporal hint and leaves the L2 to the A
  // rows every tile re-reads: 64 x 2112 x 7168 in 10.4 against 10.7 us, the
  // 16-expert masked workload 2-3 % faster.  Where tile rows share B (the
  // large shapes) the hint costs 17-19 %, so it stays off there.
  p.b_stream = p.tiles_m == 1 ? 1 : 0;
  // grouped raster height in tiles: 4 measured 1-2 % ahead of 8 and 16 on the
  // large dense and contiguous shapes (DG_GROUP_M overrides it for sweeps)
  p.group_m = 4;
  if (const char* e = getenv("DG_GROUP_M")) p.group_m = atoi(e) > 0 ? atoi(e) : 4;
}

// The launch grid is 32-bit: the output tiles (times a split count of up to
// 8) must fit it.
int set_num_tiles(dg::GemmParams& p, long long groups) {
  const long long t = groups * p.tiles_m * (long long)p.tiles_n;
  if (t > (1LL << 27)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many output tiles (%lld)", t);
  p.num_tiles = (int)t;
  return DG_OK;
}

int check_k_n(int n, int k) {
  if (n < 1) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 1 (got %d)", n);
  if (k < 128 || k % 128 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 128 (got %d)", k);
  if ((long long)n * k > 0xFFFFFFFFLL)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "one B operand must stay below 4 GiB (n*k = %lld)", (long long)n * k);
  return DG_OK;
}

// The kernels address one operand matrix (one expert's, for the grouped
// layouts) with 32-bit byte offsets.
int check_rows(long long rows, int k) {
  if (rows * k > 0xFFFFFFFFLL)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "one A operand must stay below 4 GiB (rows*k = %lld)", rows * k);
  return DG_OK;
}

// Large tiles (256 x 256 for BF16 and FP4, 128 x 256 two per CU for FP8)
// while 256 x 256 tiles alone would keep more than half the CUs busy, so
// that no split-K is needed; below that, 128 x 128 tiles (two per CU, split
// over K when still too few) finish sooner.  The
// N- and M-shards of the large GEMM over 8 GPUs, 4096 x 896 x 16384 and
// 512 x 7168 x 16384, run in 83-90 us against 107 us for 256 x 256 tiles
// split 4 ways; 2048 x 7168 x 16384 (224 big tiles) keeps 256 x 256 tiles,
// 258 against 288 us.
bool big_tiles_enough(int m, int n, const DeviceInfo* info) {
  return 2 * (long long)((m + 255) / 256) * ((n + 255) / 256) > info->cus;
}

// Split count of a dense launch of num_tiles tiles over kb_count 128-byte K
// slabs (1: no split), and the slabs of each split.
//
// K is split over workgroups when the tiles alone cannot fill the GPU's
// workgroup slots: up to two resident workgroups per CU (one for the
// configurations that fit only one).  Decode-shaped calls are bound by HBM
// latency more than by bandwidth, and two workgroups per CU keep more loads
// in flight than one (64 x 2112 x 7168: 7 splits of 8 slabs of 64 x 32 tiles,
// 462 workgroups); mid-sized shapes with too few tiles gain the same way
// (4096 x 896 x 16384 in 128 x 128 tiles: 2 splits, 83 against 115 us).
// DG_SPLIT_K=<n> pins the count (for sweeps).
int dense_splits(const Config* c, int num_tiles, int kb_count, const DeviceInfo* info, int* split_slabs) {
  int splits = 1;
  const int slots = (per_cu(c) >= 2 ? 2 : 1) * info->cus;
  if (const char* e = getenv("DG_SPLIT_K")) splits = atoi(e);
  else if (c->sched != dg::kPingPong && num_tiles * 2 <= slots && kb_count >= 4) {
    splits = slots / num_tiles;
    // no more splits than it takes to shorten the longest one
    while (splits > 1 && (kb_count + splits - 2) / (splits - 1) == (kb_count + splits - 1) / splits) --splits;
    const int min_split_slabs = 2;
    if (splits > kb_count / min_split_slabs) splits = kb_count / min_split_slabs;
    if (splits > 8) splits = 8;  // partial-tile traffic grows with the count
  }
  *split_slabs = kb_count;
  if (splits <= 1) return 1;
  const int per = (kb_count + splits - 1) / splits;
  *split_slabs = per;
  return (kb_count + per - 1) / per;  // no empty splits
}

// The default configuration of a dense call (the rules and their
// measurements are next to big_tiles_enough and in the config table).
// kb: K in 128-byte slabs (k / 128 for fp8, 2 k / 128 for bf16, k / 256 for fp4).
const Config* dense_default_config(int dtype, int m, int n, int kb, const DeviceInfo* info) {
  const bool mid = m <= 256 || n <= 256 || !big_tiles_enough(m, n, info);
  // Few 128 x 128 tiles: smaller tiles (four or more workgroups per CU), or
  // a third stage, keep more loads in flight per CU than split-K of the
  // 128 x 128 tile alone does.
  const long long t128 = (long long)((m + 127) / 128) * ((n + 127) / 128);
  const bool few = mid && m <= 256 && t128 <= 64;
  switch (dtype) {
    case dg::kBf16:
      // kb counts 64-value slabs here.  From a sweep of the pages' shapes
      // (medians, us): m <= 64 keeps 64 x 32 up to N 4096 and at N 7168 with
      // K 2048 (12.5 against 13.5), 64 x 64 beyond (64 x 7168 x 16384: 58.9
      // against 70.2; 64 x 32768 x 512: 9.3 against 10.9); m <= 128 with K up
      // to 2048 takes 64 x 64 (128 x 32768 x 512: 13.6 against 20.4 for
      // 128 x 128; 128 x 24576 x 1536: 28.5 against 32.7; 128 x 7168 x 2048:
      // 16.7 against 24.4).
      if (m <= 64) {
        const bool narrow = n <= 4096 || (n <= 8192 && kb <= 32);
        // two slabs per step (four stages): 16 x 2112 x 7168 in 12.9 against
        // 14.7 us, 64 x 4096 x 7168 18.7 against 21.7, 64 x 7168 x 2048 12.5
        // against 13.9, 64 x 2112 x 7168 level (13.5); three slabs per step
        // lost at 64 x 2112 x 7168 (14.0)
        return find_config(narrow ? "bf16_64x32_w4_s4_pair" : "bf16_64x64_w4_s3", dg::kDense, dg::kBf16);
      }
      if (few && n <= 1024) return find_config("bf16_64x32_w4_s4_pair", dg::kDense, dg::kBf16);
      if ((few && n <= 4096) || (m <= 128 && kb <= 32)) return find_config("bf16_64x64_w4_s3", dg::kDense, dg::kBf16);
      return find_config(mid ? "bf16_128x128_w4_s2" : "bf16_256x256_w8_s2", dg::kDense, dg::kBf16);
    case dg::kFp4:
      // kb counts 256-value slabs here.  From the same sweep: m <= 64 keeps
      // 64 x 32 at N 2112 and at N up to 8192 with K up to 2048, 64 x 64
      // elsewhere (64 x 7168 x 16384: 20.9 against 24.9; 64 x 24576 x 1536:
      // 9.5 against 10.4).  m <= 128 with up to 64 tiles takes 64 x 32 at N up
      // to 4096 with K up to 7168 and at N up to 8192 with K up to 2048
      // (128 x 7168 x 2048: 9.4 against 10.6 for 64 x 64; 128 x 2112 x 7168:
      // 11.9 against 12.7); longer K keeps 64 x 64 (128 x 7168 x 16384: 32.8
      // against 41.4).  With K up to 2048 over more tiles 64 x 64 wins
      // (128 x 24576 x 1536: 10.9 against 17.8 for 128 x 128).
      if (m <= 64) {
        const bool narrow = n <= 2112 || (n <= 8192 && kb <= 8);
        // three slabs per step (six stages), as for fp8: 64 x 2112 x 7168 in
        // 8.62 against 8.85 us, 16 x 2112 x 7168 8.52 against 8.81, 64 x 7168
        // x 2048 7.07 against 7.44 (back to back)
        // wider N or longer K: 64 x 64 with two slabs per step (four stages):
        // 64 x 7168 x 16384 in 19.7 against 21.4 us, 64 x 24576 x 1536 9.05
        // against 9.63, 128 x 7168 x 4096 11.8 against 13.5
        return find_config(narrow ? "fp4_64x32_w4_s6_triple" : "fp4_64x64_w4_s4_pair", dg::kDense, dg::kFp4);
      }
      if ((few && n <= 1024) || (m <= 128 && t128 <= 64 && (n <= 4096 ? kb <= 28 : n <= 8192 && kb <= 8)))
        return find_config("fp4_64x32_w4_s6_triple", dg::kDense, dg::kFp4);
      if (few || (mid && t128 <= 72 && n >= 1024) || (m <= 128 && kb <= 8))
        return find_config("fp4_64x64_w4_s4_pair", dg::kDense, dg::kFp4);
      return find_config(mid ? "fp4_128x128_w4_s2" : "fp4_256x256_w8_s2", dg::kDense, dg::kFp4);
    default: {
      // m <= 64: 64 x 32 tiles up to N 4096, and up to N 8192 while K is
      // short (at most 16 slabs): 64 x 7168 x 2048 in 10.0 against 11.3 us
      // for 64 x 64, which leads at long K (64 x 7168 x 16384: 34.0 against
      // 41.0 us) and at N 24576 (13.0 against 13.5 us).  The 64 x 32 tile
      // consumes three slabs per barrier step (six stages): its steps are
      // latency chains, not bandwidth (back to back, us, one slab per step
      // against three: 64 x 2112 x 7168 10.50 / 10.07, 32 x 2112 x 7168
      // 10.33 / 9.56, 64 x 4096 x 7168 14.18 / 12.88, 64 x 576 x 7168
      // 8.45 / 7.92, 64 x 7168 x 2048 9.33 / 8.88, 64 x 512 x 1024 5.06 /
      // 4.94).
      if (m <= 64)
        return find_config(n <= 4096 || (kb <= 16 && n <= 8192) ? "dense_64x32_w4_s6_triple" : "dense_64x64_w4_s4_pair",
                           dg::kDense);
      // large: the 128 x 256 one-B-buffer tile, two workgroups per CU.  Medians
      // of five alternating runs against 256 x 256: 4096 x 7168 x 16384 467
      // against 489 us, 2048 x 7168 x 16384 248 against 260, 4096 x 4096 x
      // 16384 264 against 266, 4096 x 8192 x 16384 522 against 516.
      if (!mid) return find_config("dense_128x256_w4_s2_sb", dg::kDense);
      // few tiles; at m <= 128 with short K also up to 128 of them (128 x
      // 12288 x 1536: 64 x 64 in 11.5 against 15.4 us for 128 x 128 with
      // three stages and 20.7 us with two).  64 x 32 tiles where N is small,
      // or at m <= 128 with up to 64 tiles and K up to 16 slabs: 128 x 7168 x
      // 1536 in 10.0 against 11.4 us, 128 x 2112 x 1536 in 9.8 against 11.1,
      // 128 x 7168 x 2048 in 11.3 against 11.7; with more tiles 64 x 64 leads
      // (128 x 16384 x 1024: 10.0 against 12.3 us), and at long K too (128 x
      // 2112 x 7168: 13.8 against 15.5 us).
      if (few || (m <= 128 && t128 <= 128 && kb <= 12)) {
        const bool narrow = n <= 1024 || (m <= 128 && t128 <= 64 && kb <= 16);
        // multi-slab steps here too: 128 x 2112 x 1024 in 5.96 against 6.20 us
        // (64 x 32, three per step); 64 x 64 with two per step and four
        // stages against three stages one per step: 128 x 16384 x 1024 9.00
        // against 9.99, 128 x 12288 x 1536 11.69 against 12.37, 64 x 24576 x
        // 1536 12.53 against 12.89, 64 x 7168 x 16384 32.6 against 33.0,
        // 64 x 8192 x 7168 18.5 against 18.9 us
        return find_config(narrow ? "dense_64x32_w4_s6_triple" : "dense_64x64_w4_s4_pair", dg::kDense);
      }
      if (t128 <= 72 && n >= 1024) return find_config("dense_128x128_w4_s3", dg::kDense);
      // short K (at most 12 slabs) where the two-per-CU tile would be split
      // over K: three stages unsplit instead.  128 x 24576 x 1536 in 16.7
      // against 22.7 us, 128 x 32768 x 512 in 9.2 against 19.2 us.
      if (kb <= 12 && t128 <= info->cus) return find_config("dense_128x128_w4_s3", dg::kDense);
      return find_config("dense_128x128_w4_s2", dg::kDense);
    }
  }
}

// The configuration a dense call uses: DG_FORCE_CONFIG when it names one of
// this dtype's dense configurations, else the default.
int dense_config(int dtype, int m, int n, int kb, const DeviceInfo* info, const Config** out) {
  if (int s = forced_config(dg::kDense, out, dtype)) return s;
  if (!*out) *out = dense_default_config(dtype, m, n, kb, info);
  if (!*out) return fail(DG_ERR_INTERNAL, "no dense configuration for dtype %d", dtype);
  return DG_OK;
}

// Dense launch with the split-K choice, shared by the fp8, bf16 and fp4 entry
// points; k_bytes is K in bytes (one per fp8 value, two per bf16 value, half
// per fp4 value) and scale_slabs the number of 128-wide scale slabs of K.
int launch_dense(const Config* c, dg::GemmParams& p, int dev, const DeviceInfo* info, int m, int n, int k_bytes,
                 int scale_slabs, dg_stream_t stream, const WsSource& ws = WsSource{}) {
  if (int s = ensure_kernel_attributes()) return s;
  p.num_groups = 1;
  fill_common(p, *c, m, n, k_bytes);
  p.sk_count = scale_slabs;
  if (int s = set_num_tiles(p, 1)) return s;
  p.splits = dense_splits(c, p.num_tiles, p.kb_count, info, &p.split_slabs);
  if (p.splits > 1) {
    if (c->sched == dg::kPingPong)
      return fail(DG_ERR_INVALID_ARGUMENT, "configuration %s does not support split-K", c->name);
    if ((size_t)p.num_tiles > kCounterInts)
      return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many tiles for split-K (%d)", p.num_tiles);
    if ((long long)p.num_tiles * p.splits > 0x7FFFFFFFLL)
      return fail(DG_ERR_UNSUPPORTED_SHAPE, "split-K grid too large (%d x %d)", p.num_tiles, p.splits);
    const size_t part = (size_t)p.num_tiles * p.splits * c->bm * c->bn * sizeof(float);
    WsView v;
    if (int s = get_workspace(ws, dev, (hipStream_t)stream, part, p.num_tiles, &v)) return s;
    p.ws_partial = (float*)v.partial;
    p.ws_count = v.counters;
  }
  return launch(*c, p, p.num_tiles * p.splits, (hipStream_t)stream);
}

// ---- skinny-M plan: the stream-K partition of a dense fp8 call with m <= 64
struct SkinnyPlan {
  const SkinnyConfig* c = nullptr;
  int tiles_n = 0, grid = 0, per = 0, rem = 0, max_contrib = 0;
  size_t ws_bytes = 0;  // 0: no tile is cut between workgroups
};

// Workgroups: one per CU when there are enough units (a unit is one 128-wide
// K slab of one 64 x BN tile), each taking an equal contiguous run of at most
// NW units (one per wave); more workgroups when the runs would be longer than
// NW.  A tile cut by run boundaries is added up by its last contributor, which
// reads at most dg::kSkinnyMaxContrib partials, so runs are at least
// ceil(KB / (dg::kSkinnyMaxContrib - 1)) units.  Returns false when the shape
// does not fit these rules.
bool skinny_plan(const SkinnyConfig* c, int m, int n, int kb, const DeviceInfo* info, SkinnyPlan* out) {
  if (m < 1 || m > 64) return false;
  const long long tiles_n = (n + c->bn - 1) / c->bn;
  const long long units = tiles_n * kb;
  if (units > (1LL << 30) || tiles_n > (long long)kCounterInts) return false;
  long long grid = units < info->cus ? units : info->cus;
  const long long need = (units + c->units_per_wg() - 1) / c->units_per_wg();  // runs of at most NW * UPW units
  if (grid < need) grid = need;
  const long long per_min = (kb + dg::kSkinnyMaxContrib - 2) / (dg::kSkinnyMaxContrib - 1);
  if (per_min > c->units_per_wg()) return false;
  if (grid > units / per_min) grid = units / per_min;
  if (grid < need || grid < 1) return false;
  SkinnyPlan pl;
  pl.c = c;
  pl.tiles_n = (int)tiles_n;
  pl.grid = (int)grid;
  pl.per = (int)(units / grid);
  pl.rem = (int)(units % grid);
  const int mc = (kb + pl.per - 1) / pl.per + 1;
  pl.max_contrib = mc < dg::kSkinnyMaxContrib ? mc : dg::kSkinnyMaxContrib;
  bool cut = false;
  for (int L = 1; L < pl.grid && !cut; ++L) cut = ((long long)L * pl.per + (L < pl.rem ? L : pl.rem)) % kb != 0;
  pl.ws_bytes = cut ? (size_t)tiles_n * pl.max_contrib * 64 * c->bn * sizeof(float) : 0;
  *out = pl;
  return true;
}

// The skinny configuration a dense fp8 call uses (nullptr: the tiled kernels):
// only DG_FORCE_CONFIG naming a skinny configuration (then m must be at most
// 64).  The skinny kernel used to be the default for m <= 16 (N 2112 K 7168
// in 9.4-9.6 against 10.9-11.2 us for the tiled split-K kernel of the time);
// since the tiled 64 x 32 kernel takes three slabs per step it is ahead at
// every m <= 16 shape measured (back to back, us, skinny / tiled): 8 x 2112
// x 7168 9.87 / 9.52, 1 x 2112 x 7168 9.82 / 9.38, 16 x 2112 x 7168 10.04 /
// 9.52, 8 x 7168 x 2048 9.09 / 8.28, 16 x 7168 x 2048 9.28 / 8.31, 4 x 576
// x 7168 11.23 / 7.75, 16 x 4096 x 7168 17.16 / 11.47.
int skinny_config(int m, int n, int kb, const DeviceInfo* info, SkinnyPlan* plan) {
  plan->c = nullptr;
  const char* e = getenv("DG_FORCE_CONFIG");
  if (e && *e) {
    const SkinnyConfig* c = find_skinny(e);
    if (!c) return DG_OK;  // a tiled configuration (or an unknown name, reported by dense_config)
    if (!skinny_plan(c, m, n, kb, info, plan))
      return fail(DG_ERR_INVALID_ARGUMENT, "configuration %s does not take m=%d n=%d k=%d", e, m, n, kb * 128);
    return DG_OK;
  }
  (void)m; (void)n; (void)kb; (void)info;
  return DG_OK;
}

int launch_skinny(const SkinnyPlan& pl, const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                  uint16_t* d, int m, int n, int k, int dev, dg_stream_t stream, const WsSource& ws = WsSource{}) {
  if (int s = ensure_kernel_attributes()) return s;
  dg::SkinnyParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d;
  p.m = m; p.n = n; p.k = k;
  p.kb_count = k / 128;
  p.sfa_ld = sfa_ld(m);
  p.tiles_n = pl.tiles_n;
  p.per = pl.per;
  p.rem = pl.rem;
  p.max_contrib = pl.max_contrib;
  if (pl.ws_bytes > 0) {
    WsView v;
    if (int s = get_workspace(ws, dev, (hipStream_t)stream, pl.ws_bytes, pl.tiles_n, &v)) return s;
    p.ws_partial = (float*)v.partial;
    p.ws_count = v.counters;
  }
  const SkinnyConfig& c = *pl.c;
  if (log_enabled())
    fprintf(stderr, "[dg] %s m=%d n=%d k=%d grid=%d threads=%d smem=%d per=%d rem=%d contrib=%d ws=%zu\n", c.name, m,
            n, k, pl.grid, c.threads(), c.smem(), pl.per, pl.rem, pl.max_contrib, pl.ws_bytes);
  void* args[] = {&p};
  const hipError_t e = launch_gemm_kernel(c.fn, dim3(pl.grid), c.threads(), args, c.smem(), (hipStream_t)stream);
  if (e != hipSuccess) return fail(DG_ERR_HIP, "launch of %s failed: %s", c.name, hipGetErrorString(e));
  return ok();
}

int quantize_a(const void* kernel, const float* x, uint8_t* q, float* sfa, int m, int k, dg_stream_t stream) {
  if (!x || !q || !sfa) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (k < 128 || k % 128 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 128 (got %d)", k);
  if (!aligned16(x) || !aligned16(q) || !aligned16(sfa))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const int ld = sfa_ld(m);
  const long long units = (long long)ld * ((k / 128 + 1) / 2);
  const long long grid = (units + 3) / 4;
  if (grid > 0x7fffffffLL) return fail(DG_ERR_UNSUPPORTED_SHAPE, "matrix too large");
  void* args[] = {&x, &q, &sfa, &m, &k, (void*)&ld};
  hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)grid), dim3(256), args, 0, (hipStream_t)stream);
  if (e != hipSuccess) return fail(DG_ERR_HIP, "quant_a launch failed: %s", hipGetErrorString(e));
  return ok();
}

int quantize_b(const void* kernel, const float* x, uint8_t* q, float* sfb, int n, int k, dg_stream_t stream) {
  if (!x || !q || !sfb) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (n < 0) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 0 (got %d)", n);
  if (k < 128 || k % 128 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 128 (got %d)", k);
  if (!aligned16(x) || !aligned16(q) || !aligned16(sfb))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (n == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const long long grid = (long long)((n + 127) / 128) * (k / 128);
  if (grid > 0x7fffffffLL) return fail(DG_ERR_UNSUPPORTED_SHAPE, "matrix too large");
  void* args[] = {&x, &q, &sfb, &n, &k};
  hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)grid), dim3(256), args, 0, (hipStream_t)stream);
  if (e != hipSuccess) return fail(DG_ERR_HIP, "quant_b launch failed: %s", hipGetErrorString(e));
  return ok();
}


// The dense fp8 call, with the split-K workspace of the calling stream or,
// for the allocation-free entry point, the static scratch.
int fp8_gemm(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d, int m, int n, int k,
             dg_stream_t stream, bool use_scratch) {
  if (!a || !sfa || !b || !sfb || !d) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (int s = check_k_n(n, k)) return s;
  if (int s = check_rows(m, k)) return s;
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(d))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  WsSource ws;
  if (use_scratch)
    if (int s = scratch_address(dev, &ws.fixed)) return s;
  SkinnyPlan sp;
  if (int s = skinny_config(m, n, k / 128, info, &sp)) return s;
  if (sp.c) return launch_skinny(sp, a, sfa, b, sfb, d, m, n, k, dev, stream, ws);
  const Config* c;
  if (int s = dense_config(dg::kFp8, m, n, k / 128, info, &c)) return s;
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d;
  return launch_dense(c, p, dev, info, m, n, k, k / 128, stream, ws);
}

// ---- 4-bit weights with group scales (w4_kernel.h)

int check_w4(int n, int k, int group, int format, const void* zeros) {
  if (format != DG_W4_E2M1 && format != DG_W4_U4)
    return fail(DG_ERR_INVALID_ARGUMENT, "unknown 4-bit format %d", format);
  if ((format == DG_W4_U4) != (zeros != nullptr))
    return fail(DG_ERR_INVALID_ARGUMENT, "zeros go with DG_W4_U4 and with it only");
  if (n < 1) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 1 (got %d)", n);
  if (group != 32 && group != 64 && group != 128)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "group must be 32, 64 or 128 (got %d)", group);
  if (k > (1 << 23)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be at most 2^23 (got %d)", k);  // 32-bit offsets
  if (k < group || k % group != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of the group of %d (got %d)", group, k);
  return DG_OK;
}

// How a product is launched: workgroups of 16 weight rows by up to 16 rows of a
// whose waves split K, or tiles of 128 weight rows by 32 or 64 rows of a and K
// in splits.
struct W4Plan {
  const char* name;
  const void* fn;
  dim3 grid;
  int threads, smem;
  size_t partial_bytes;  // split tiles, 0 if K is not split
  int tiles;
};

template <int FMT, int GROUP, bool WHOLE>
W4Plan w4_plan(int m, int n, int k, const DeviceInfo* info, const char* way) {
  const int units = (k + 127) / 128;
  // 16 x 16 tiles up to 16 rows, and beyond while each CU has no more than about
  // 100 units of them (us, 16 x 16 / larger tiles, units per CU: 64 x 512 x 1024
  // 3.3 / 8.8 with 4, 64 x 4096 x 1024 4.9 / 8.9 with 32, 24 x 7168 x 2048 8.4 /
  // 8.5 with 56, 48 x 2112 x 7168 11.2 / 15.5 with 87, 32 x 4096 x 7168 13.4 /
  // 12.5 and 64 x 7168 x 2048 12.6 / 10.8 with 112, 64 x 4096 x 7168 21.8 / 18.0
  // with 224).
  const long long small_tiles = (long long)((n + 15) / 16) * ((m + 15) / 16);
  bool small = m <= 16 || small_tiles * units <= 100LL * info->cus;
  if (way) small = way == kW4RowsName;
  if (small) {
    // 8 waves for up to one and a half workgroups per CU, then 4, which leave
    // more of them side by side (us, 4 / 8 / 16 waves: 1 x 2112 x 7168 5.2 / 4.7
    // / 4.9, 1 x 4096 x 7168 6.1 / 5.9 / 6.2, 8 x 4096 x 7168 8.9 / 7.7 / 8.0,
    // 1 x 7168 x 16384 12.6 / 14.1 / 15.3, 1 x 16384 x 2048 6.7 / 7.6 / 12.7);
    // 4 also where 8 would have two units each or fewer (1 x 512 x 1024 3.1 /
    // 3.3 / 3.6).  With more than 8 rows always 8, as there is more to compute
    // than to load (16 x 7168 x 16384, groups of 32: 33.5 / 27.1).
    const dim3 grid((n + 15) / 16, (m + 15) / 16);
    const int waves = units >= 16 && (m > 8 || 2LL * grid.x <= 3LL * info->cus) ? 8 : 4;
    // rows of a staged: no more than needed (8 waves; 4 / 8 / 16 rows: 1 x 4096 x
    // 7168 6.0 / 6.4 / 7.3; 4 x 4096 x 7168 7.6 / 7.7 / 8.5; 5 x 2112 x 7168 - /
    // 5.2 / 6.3)
    if (m <= 4)
      return {kW4RowsName, reinterpret_cast<const void*>(&dg::w4_rows_kernel<FMT, GROUP, 2, 4, WHOLE>), grid, waves * 64,
              dg::w4_rows_smem<FMT, GROUP, 2, 4, WHOLE>(waves), 0, 0};
    if (m <= 8)
      return {kW4RowsName, reinterpret_cast<const void*>(&dg::w4_rows_kernel<FMT, GROUP, 1, 8, WHOLE>), grid, waves * 64,
              dg::w4_rows_smem<FMT, GROUP, 1, 8, WHOLE>(waves), 0, 0};
    return {kW4RowsName, reinterpret_cast<const void*>(&dg::w4_rows_kernel<FMT, GROUP, 1, 16, WHOLE>), grid, waves * 64,
            dg::w4_rows_smem<FMT, GROUP, 1, 16, WHOLE>(waves), 0, 0};
  }
  // (at m = 17 and 32 tiles of 64 rows take 16.7 us for 4096 x 7168 against 12.9
  // and 27.3 for 7168 x 16384 against 20.0)
  const int rows = m <= 32 ? 32 : 64;
  const int tiles_n = (n + 127) / 128, tiles_m = (m + rows - 1) / rows;
  const long long tiles = (long long)tiles_n * tiles_m;
  // At least four units a split and at most 8 splits (the last of them adds all
  // up: 64 x 2112 x 7168 15.1 us with 8, 18.6 with 16).  Within that, as many as
  // give each CU one workgroup or, where those have many units, two.  One takes
  // about 0.6 us a unit, two side by side 1.0 us for a unit of each and 2.5 us
  // more (us, one / two per CU: 128 x 2112 x 7168 15.4 / 19.9, 128 x 4096 x 7168
  // 16.8 / 20.6, 48 x 5120 x 5120 14.9 / 16.8, 64 x 10240 x 4096 18.7 / 19.5;
  // 200 x 2112 x 7168 31.5 / 29.4, 96 x 7168 x 7168 35.1 / 31.6, 128 x 7168 x
  // 16384 47.7 / 43.6, 512 x 2112 x 7168 39.8 / 31.3).  Other shapes, against two
  // per CU always: 70 x 2112 x 16384 28.1 for 34.9, 160 x 1536 x 8192 17.7 for
  // 22.0, 40 x 6144 x 6144 15.1 for 16.1; near the border u4 can lose (24 x 14336
  // x 4096 16.5 for 15.5, 80 x 8192 x 4096 23.2 for 22.0).
  const long long most = units / 4 < 8 ? units / 4 : 8;
  const auto fit = [&](long long per_cu) {
    const long long s = per_cu * info->cus / tiles;
    return s < 1 || most < 1 ? 1 : s < most ? s : most;
  };
  const long long one = fit(1), two = fit(2);
  const long long of_one = (units + one - 1) / one, of_two = (units + two - 1) / two;
  long long splits = tiles > info->cus || 6 * of_one > 10 * of_two + 25 ? two : one;
  if (const char* e = getenv("DG_SPLIT_K")) splits = atoi(e) < units ? atoi(e) : units;
  if (splits < 1 || tiles > (long long)kCounterInts) splits = 1;
  return {kW4TileName,
          rows == 32 ? reinterpret_cast<const void*>(&dg::w4_tile_kernel<FMT, GROUP, 2, WHOLE>)
                     : reinterpret_cast<const void*>(&dg::w4_tile_kernel<FMT, GROUP, 4, WHOLE>),
          dim3(tiles_n, (unsigned)splits, tiles_m), 256, 0,
          splits > 1 ? (size_t)tiles * splits * rows * 128 * sizeof(float) : 0, (int)tiles};
}

template <int FMT, int GROUP>
W4Plan w4_plan(int m, int n, int k, const DeviceInfo* info, const char* way) {
  if constexpr (GROUP == 128) return w4_plan<FMT, GROUP, true>(m, n, k, info, way);
  return k % 128 == 0 ? w4_plan<FMT, GROUP, true>(m, n, k, info, way) : w4_plan<FMT, GROUP, false>(m, n, k, info, way);
}

template <int FMT>
W4Plan w4_plan(int m, int n, int k, int group, const DeviceInfo* info, const char* way) {
  return group == 32   ? w4_plan<FMT, 32>(m, n, k, info, way)
         : group == 64 ? w4_plan<FMT, 64>(m, n, k, info, way)
                       : w4_plan<FMT, 128>(m, n, k, info, way);
}

// `way`: kW4RowsName, kW4TileName, or null for the rule's choice
W4Plan w4_plan(int m, int n, int k, int group, int format, const DeviceInfo* info, const char* way) {
  return format == DG_W4_E2M1 ? w4_plan<dg::kW4E2m1>(m, n, k, group, info, way)
                              : w4_plan<dg::kW4U4>(m, n, k, group, info, way);
}

template <int FMT, bool BF16>
const void* w4_quant_fn(int group) {
  return group == 32   ? reinterpret_cast<const void*>(&dg::w4_quant_kernel<FMT, 32, BF16>)
         : group == 64 ? reinterpret_cast<const void*>(&dg::w4_quant_kernel<FMT, 64, BF16>)
                       : reinterpret_cast<const void*>(&dg::w4_quant_kernel<FMT, 128, BF16>);
}

template <int FMT>
const void* w4_dequant_fn(int group) {
  return group == 32   ? reinterpret_cast<const void*>(&dg::w4_dequant_kernel<FMT, 32>)
         : group == 64 ? reinterpret_cast<const void*>(&dg::w4_dequant_kernel<FMT, 64>)
                       : reinterpret_cast<const void*>(&dg::w4_dequant_kernel<FMT, 128>);
}

int launch_plain(const char* what, const void* fn, dim3 grid, int threads, void** args, dg_stream_t stream, int smem = 0,
                 bool gemm = false) {
  if (log_enabled())
    fprintf(stderr, "[dg] %s grid=%ux%ux%u threads=%d\n", what, grid.x, grid.y, grid.z, threads);
  const hipError_t e = gemm ? launch_gemm_kernel(fn, grid, threads, args, smem, (hipStream_t)stream)
                            : hipLaunchKernel(fn, grid, dim3(threads), args, smem, (hipStream_t)stream);
  if (e != hipSuccess) return fail(DG_ERR_HIP, "launch of %s failed: %s", what, hipGetErrorString(e));
  return ok();
}

// ---- 8-bit key/value cache (kv8_kernel.h)

// Arrays without elements may be null: no pool, no table, no sequences.
int check_cache(const void* k_codes, const void* v_codes, const void* k_scales, const void* v_scales, const void* table,
                int batch, int h_kv, int d, int block, int num_blocks, int max_blocks, dg::Kv8Cache* c) {
  if ((num_blocks != 0 && (!k_codes || !v_codes || !k_scales || !v_scales)) || (batch != 0 && max_blocks != 0 && !table))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (h_kv < 1 || h_kv > 32767) return fail(DG_ERR_INVALID_ARGUMENT, "h_kv must be 1..32767 (got %d)", h_kv);
  if (num_blocks < 0 || max_blocks < 0) return fail(DG_ERR_INVALID_ARGUMENT, "block counts must be >= 0");
  if (d != 64 && d != 128 && d != 256)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "head dimension must be 64, 128 or 256 (got %d)", d);
  int log2 = 4;
  while (log2 < 7 && (1 << log2) != block) ++log2;
  if ((1 << log2) != block)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "block must be 16, 32, 64 or 128 tokens (got %d)", block);
  if (((long long)max_blocks << log2) > (1LL << 30))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "a sequence's table may span at most 2^30 tokens");
  if (!aligned16(k_codes) || !aligned16(v_codes) || (reinterpret_cast<uintptr_t>(k_scales) & 3u) ||
      (reinterpret_cast<uintptr_t>(v_scales) & 3u) || (reinterpret_cast<uintptr_t>(table) & 3u))
    return fail(DG_ERR_MISALIGNED, "codes must be 16-byte aligned, scales and block table 4-byte");
  c->k_codes = (uint8_t*)k_codes;
  c->v_codes = (uint8_t*)v_codes;
  c->k_scales = (float*)k_scales;
  c->v_scales = (float*)v_scales;
  c->table = (const int32_t*)table;
  c->h_kv = h_kv;
  c->block = block;
  c->block_log2 = log2;
  c->num_blocks = num_blocks;
  c->max_blocks = max_blocks;
  return DG_OK;
}

int check_packed(const void* x, int64_t stride, int heads, int d, const char* name) {
  if (!aligned16(x)) return fail(DG_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
  if (stride < (int64_t)heads * d || stride % 8 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: the stride between tokens must be a multiple of 8 elements and at least "
                "heads * d (got %lld)", name, (long long)stride);
  return DG_OK;
}

int check_batch(int batch, int total, int most) {
  if (batch < 0 || total < 0 || most < 0)
    return fail(DG_ERR_INVALID_ARGUMENT, "batch, token counts and the longest sequence must be >= 0");
  if (batch > 65535) return fail(DG_ERR_UNSUPPORTED_SHAPE, "at most 65535 sequences (got %d)", batch);
  return DG_OK;
}

// Workgroups that share an attention call: one per CU.  Its four waves keep 64
// KB of codes in flight, enough for HBM, and fewer shares leave fewer parts to
// join (us, one / two per CU: 4 x 65536 keys, 64 / 8 heads of 128 101 / 108; 32 x
// 4096, 32 / 8 heads of 128 44 / 51, of 64 27 / 29; 4 x 8192, 16 / 4 heads of 256
// 22 / 38).
// Each leaves at most two unfinished 16-row tiles.
int kv8_workers(const DeviceInfo* info) { return info->cus; }
size_t kv8_part_floats(int workers, int d) { return (size_t)workers * 2 * 16 * (d + 2); }

// ---- latent attention (latent_kernel.h)

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The scale in units of log2, and not 0: 0 times what is masked would be no mask.
float latent_scale(float scale) {
  const float s = scale * 1.44269504088896340736f;
  return s > 1.17549435e-38f ? s : 1.17549435e-38f;
}

int check_latent_dim(int latent) {
  if (latent != 256 && latent != 512)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "the latent must have 256 or 512 values (got %d)", latent);
  return DG_OK;
}

// Arrays without elements may be null: no pool, no table, no sequences.
int check_latent_cache(const void* latent, const void* rope, const void* scales, const void* table, int batch,
                       int latent_dim, int block, int num_blocks, int max_blocks, dg::LatentCache* c) {
  if (int s = check_latent_dim(latent_dim)) return s;
  if ((num_blocks != 0 && (!latent || !rope)) || (batch != 0 && max_blocks != 0 && !table))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (num_blocks < 0 || max_blocks < 0) return fail(DG_ERR_INVALID_ARGUMENT, "block counts must be >= 0");
  int log2 = 4;
  while (log2 < 7 && (1 << log2) != block) ++log2;
  if ((1 << log2) != block)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "block must be 16, 32, 64 or 128 tokens (got %d)", block);
  if (((long long)max_blocks << log2) > (1LL << 30))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "a sequence's table may span at most 2^30 tokens");
  if (!aligned16(latent) || !aligned16(rope) || !aligned16(scales) || !aligned4(table))
    return fail(DG_ERR_MISALIGNED, "cache arrays must be 16-byte aligned, the block table 4-byte");
  c->latent = (uint8_t*)latent;
  c->rope = (uint16_t*)rope;
  c->scales = (float*)scales;
  c->table = (const int32_t*)table;
  c->block = block;
  c->block_log2 = log2;
  c->num_blocks = num_blocks;
  c->max_blocks = num_blocks == 0 ? 0 : max_blocks;  // no blocks: no tokens, whatever the lengths say
  return DG_OK;
}

// Rows of heads with strides of their own: from token to token and from head to
// head, either of which may be 0, one row for all; rows that are written have to
// pass check_apart too.
int check_strided(const void* x, int64_t stride, int64_t head_stride, int heads, int d, int unit, const char* name) {
  if ((reinterpret_cast<uintptr_t>(x) & (unit * 2 - 1)) != 0)
    return fail(DG_ERR_MISALIGNED, "%s must be %d-byte aligned", name, unit * 2);
  if (stride < 0 || head_stride < 0 || stride % unit != 0 || head_stride % unit != 0 ||
      (heads > 1 && head_stride != 0 && head_stride < d))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: strides must be multiples of %d elements, and 0 or at least %d from head "
                "to head (got %lld, %lld)", name, unit, d, (long long)stride, (long long)head_stride);
  return DG_OK;
}

// Rows that are written: no two of them may overlap, one of the strides has to step over all that the other one reaches.
int check_apart(int64_t stride, int64_t head_stride, int total, int heads, int d, const char* name) {
  const __int128 token = stride, head = head_stride;
  const bool apart = (total <= 1 || token >= d) && (heads <= 1 || head >= d) &&
                     (total <= 1 || heads <= 1 || token >= (heads - 1) * head + d || head >= (total - 1) * token + d);
  return apart ? DG_OK : fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: rows of %d tokens and %d heads overlap (strides %lld, %lld)", name,
                              total, heads, (long long)stride, (long long)head_stride);
}

// Tiles of 16 rows that a workgroup of absorbed attention takes at once: as many
// as one sequence's queries fill, up to four, if there are more than four
// 64-token steps of such tiles for each workgroup; else one, as a
// large tile's only step and part then cost more than reading the tokens again
// (us with 16 / 32 / 64 rows, bf16, latents of 512, 128 heads: 1 x 4096 20 / 30 / 32,
// 8 x 1024 23 / 28 / 33, 1 x 16384 30 / 34 / 40, 32 x 1024 35 / 35 / 38, 4 x 65536
// 244 / 148 / 112; 64 heads: 64 x 512 24 / 29 / 34; 32 heads: 1 x 8192 23 / 32, 16 x
// 8192 49 / 47; e4m3, 128 heads: 32 x up to 4096 94 / 72 / 70; 16 heads, 256 new
// of 2048 61 / 50 / 50).  How many steps there are the host knows from the table and
// the pool only, lengths being on the device: with a pool and tables much larger than
// the sequences it takes more rows than it should, and fewer where many sequences
// share a small pool's pages (us in a pool as large as the sequences / 16 times as
// large: 1 x 4096 20 / 33, 8 x 1024 23 / 33, 3 new of each of 16 x 2048 in e4m3 with 20
// heads 31 / 40; 32 x 4096 that share their pages 102, with 64 rows 66).
int latent_row_tiles(int max_q, int h_q, long long tokens, int workers, const char* forced) {
  for (int i = 0; forced && i < 3; ++i)
    if (strcmp(forced, kLatentRows[i]) == 0) return 1 << i;
  const long long rows = (long long)max_q * h_q;
  const int tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const long long each = (rows + 16 * tiles - 1) / (16 * tiles);
  return each > 0 && (tokens + 63) / 64 <= 4LL * workers / each ? 1 : tiles;
}
size_t latent_part_floats(int workers, int tiles, int latent) { return (size_t)workers * 2 * 16 * tiles * (latent + 2); }
size_t latent_part_bytes(int workers, int tiles, int latent) {
  return latent_part_floats(workers, tiles, latent) * sizeof(float) + workers * sizeof(dg::LatentCut);
}

int check_latent_rows(int max_q, int h_q) {
  if (h_q < 1 || h_q > 32767) return fail(DG_ERR_INVALID_ARGUMENT, "h_q must be 1..32767 (got %d)", h_q);
  if ((long long)max_q * h_q > (1LL << 30))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many queries per sequence (%d of %d heads)", max_q, h_q);
  return DG_OK;
}

struct LatentKernel {
  const void* fn;
  int smem;
  const void* join;
};

template <int L, bool F8, int NT>
LatentKernel latent_attn() {
  return {reinterpret_cast<const void*>(&dg::latent_attn_kernel<L, F8, NT>), dg::LatentLds<L, F8, NT>::kBytes,
          reinterpret_cast<const void*>(&dg::latent_join_kernel<L, NT>)};
}
template <int L, bool F8>
LatentKernel latent_attn(int tiles) {
  return tiles == 1 ? latent_attn<L, F8, 1>() : tiles == 2 ? latent_attn<L, F8, 2>() : latent_attn<L, F8, 4>();
}
LatentKernel latent_attn(int latent, bool f8, int tiles) {
  return latent == 512 ? (f8 ? latent_attn<512, true>(tiles) : latent_attn<512, false>(tiles))
                       : (f8 ? latent_attn<256, true>(tiles) : latent_attn<256, false>(tiles));
}

template <int D, int MT, bool SPLIT>
LatentKernel latent_expanded() {
  return {reinterpret_cast<const void*>(&dg::latent_expanded_kernel<D, MT, SPLIT>), 2 * dg::latent_expanded_step(SPLIT) * (4 * D + D),
          nullptr};
}
template <int D>
LatentKernel latent_expanded(int rows) {
  return rows == 128 ? latent_expanded<D, 2, false>() : rows == 64 ? latent_expanded<D, 1, false>()
         : rows == 32 ? latent_expanded<D, 2, true>() : latent_expanded<D, 1, true>();
}
LatentKernel latent_expanded(int d, int rows) { return d == 128 ? latent_expanded<128>(rows) : latent_expanded<64>(rows); }

std::once_flag g_latent_once[kMaxDevices];
hipError_t g_latent_err[kMaxDevices];

// These kernels take more LDS than a launch may ask for unasked, on each device.
int ensure_latent_attributes(int dev) {
  std::call_once(g_latent_once[dev], [dev]() {
    g_latent_err[dev] = hipSuccess;
    auto allow = [dev](const LatentKernel& k) {
      const hipError_t e = hipFuncSetAttribute(k.fn, hipFuncAttributeMaxDynamicSharedMemorySize, k.smem);
      if (e != hipSuccess) g_latent_err[dev] = e;
    };
    for (int latent : {256, 512})
      for (bool f8 : {false, true})
        for (int tiles : {1, 2, 4}) allow(latent_attn(latent, f8, tiles));
    for (int d : {64, 128})
      for (int rows : {16, 32, 64, 128}) allow(latent_expanded(d, rows));
  });
  if (g_latent_err[dev] != hipSuccess)
    return fail(DG_ERR_HIP, "hipFuncSetAttribute: %s", hipGetErrorString(g_latent_err[dev]));
  return DG_OK;
}

template <int L>
const void* latent_append_fn(bool f8, bool pairs) {
  return f8 ? (pairs ? reinterpret_cast<const void*>(&dg::latent_append_kernel<L, true, true>)
                     : reinterpret_cast<const void*>(&dg::latent_append_kernel<L, true, false>))
            : (pairs ? reinterpret_cast<const void*>(&dg::latent_append_kernel<L, false, true>)
                     : reinterpret_cast<const void*>(&dg::latent_append_kernel<L, false, false>));
}

template <int L>
const void* latent_gather_fn(bool f8) {
  return f8 ? reinterpret_cast<const void*>(&dg::latent_gather_kernel<L, true>)
            : reinterpret_cast<const void*>(&dg::latent_gather_kernel<L, false>);
}

}  // namespace

extern "C" {

int dg_get_m_alignment_for_contiguous_layout(void) { return 128; }

int dg_get_sfa_ld(int m) { return m < 0 ? 0 : sfa_ld(m); }

static_assert((int)DG_DTYPE_FP8 == (int)dg::kFp8 && (int)DG_DTYPE_BF16 == (int)dg::kBf16 &&
                  (int)DG_DTYPE_FP4 == (int)dg::kFp4,
              "dtype codes of the ABI and the kernels agree");

const char* dg_version(void) { return "dg-gfx950 0.1"; }

int dg_reserve_workspace(size_t bytes, dg_stream_t stream) {
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  char* base;
  if (int s = ensure_workspace(dev, (hipStream_t)stream, bytes, &base)) return s;
  return ok();
}

int dg_dense_workspace_size(int dtype, int m, int n, int k, size_t* bytes) {
  if (!bytes) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  *bytes = 0;
  int k_bytes = 0;
  switch (dtype) {
    case DG_DTYPE_FP8:
      if (k < 128 || k % 128 != 0)
        return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 128 (got %d)", k);
      k_bytes = k;
      break;
    case DG_DTYPE_BF16:
      if (k < 64 || k % 64 != 0 || k > (1 << 30))
        return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 64 (got %d)", k);
      k_bytes = 2 * k;
      break;
    case DG_DTYPE_FP4:
      if (k < 256 || k % 256 != 0)
        return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 256 (got %d)", k);
      k_bytes = k / 2;
      break;
    default:
      return fail(DG_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
  }
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (n < 1) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 1 (got %d)", n);
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  if (int s = ensure_kernel_attributes()) return s;
  if (dtype == DG_DTYPE_FP8) {
    SkinnyPlan sp;
    if (int s = skinny_config(m, n, k / 128, info, &sp)) return s;
    if (sp.c) {
      *bytes = sp.ws_bytes;
      return ok();
    }
  }
  const Config* c;
  if (int s = dense_config(dtype, m, n, k_bytes / 128, info, &c)) return s;
  const long long tiles = (long long)((m + c->bm - 1) / c->bm) * ((n + c->bn - 1) / c->bn);
  if (tiles > (1LL << 27)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many output tiles (%lld)", tiles);
  int per = 0;
  const int splits = dense_splits(c, (int)tiles, k_bytes / 128, info, &per);
  if (splits > 1) *bytes = (size_t)tiles * splits * c->bm * c->bn * sizeof(float);
  return ok();
}

int dg_profile_next_launch(void* start_event, void* stop_event) {
  g_prof_start = (hipEvent_t)start_event;
  g_prof_stop = (hipEvent_t)stop_event;
  return ok();
}

const char* dg_status_string(int status) {
  switch (status) {
    case DG_OK: return "ok";
    case DG_ERR_INVALID_ARGUMENT: return "invalid argument";
    case DG_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case DG_ERR_MISALIGNED: return "misaligned pointer";
    case DG_ERR_NO_DEVICE: return "no usable gfx950 device";
    case DG_ERR_HIP: return "HIP runtime error";
    case DG_ERR_INTERNAL: return "internal error";
    case DG_ERR_WORKSPACE: return "split-K workspace must grow during graph capture";
    default: return "unknown status";
  }
}

const char* dg_last_error_message(void) { return g_last_error.c_str(); }

int dg_fp8_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d,
                   int m, int n, int k, dg_stream_t stream) {
  return fp8_gemm(a, sfa, b, sfb, d, m, n, k, stream, false);
}

int dg_fp8_gemm_nt_noalloc(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d,
                           int m, int n, int k, dg_stream_t stream) {
  return fp8_gemm(a, sfa, b, sfb, d, m, n, k, stream, true);
}

int dg_bf16_gemm_nt(const uint16_t* a, const uint16_t* b, uint16_t* d, int m, int n, int k, dg_stream_t stream) {
  if (!a || !b || !d) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (n < 1) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 1 (got %d)", n);
  if (k < 64 || k % 64 != 0 || k > (1 << 30))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 64 (got %d)", k);
  if (int s = check_k_n(n, 2 * k)) return s;
  if (int s = check_rows(m, 2 * k)) return s;
  if (!aligned16(a) || !aligned16(b) || !aligned16(d)) return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = dense_config(dg::kBf16, m, n, 2 * k / 128, info, &c)) return s;
  dg::GemmParams p{};
  p.a = reinterpret_cast<const uint8_t*>(a);
  p.b = reinterpret_cast<const uint8_t*>(b);
  p.d = d;
  return launch_dense(c, p, dev, info, m, n, 2 * k, 0, stream);
}

int dg_fp4_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d, int m,
                   int n, int k, dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !d) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (n < 1) return fail(DG_ERR_INVALID_ARGUMENT, "n must be >= 1 (got %d)", n);
  if (k < 256 || k % 256 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 256 (got %d)", k);
  if (int s = check_k_n(n, k / 2)) return s;
  if (int s = check_rows(m, k / 2)) return s;
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(d))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = dense_config(dg::kFp4, m, n, k / 256, info, &c)) return s;
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d;
  return launch_dense(c, p, dev, info, m, n, k / 2, k / 128, stream);
}

int dg_m_grouped_fp8_gemm_nt_contiguous(const uint8_t* a, const float* sfa, const uint8_t* b,
                                        const float* sfb, uint16_t* d, const int32_t* m_indices, int m,
                                        int n, int k, int num_groups, dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !d || !m_indices)
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (num_groups < 1) return fail(DG_ERR_INVALID_ARGUMENT, "num_groups must be >= 1 (got %d)", num_groups);
  if (int s = check_k_n(n, k)) return s;
  if (m % 128 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "m must be a multiple of the 128-row alignment (got %d)", m);
  if (int s = check_rows(m, k)) return s;
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(d) ||
      (reinterpret_cast<uintptr_t>(m_indices) & 3u))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned (m_indices 4-byte)");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = forced_config(dg::kContiguous, &c)) return s;
  if (!c) {
    // 128 x 256 tiles with one B buffer (two workgroups per CU) once there
    // are enough of them to fill the GPU; 128 x 128 tiles below that, and
    // 64 x 64 tiles (more workgroups per CU) while 128 x 128 tiles would be
    // at most 128: 4 x 128 rows, N 4096, K 7168 in 49.8 against 63.7 us,
    // N 2112 in 42.9 against 59.9 us; at 256 such tiles they lose (101
    // against 72 us).
    const long long tiles = (long long)(m / 128) * ((n + 255) / 256);
    const long long t128 = (long long)(m / 128) * ((n + 127) / 128);
    c = find_config(t128 <= 128        ? "contig_64x64_w4_s3"
                    : tiles >= info->cus ? "contig_128x256_w4_s2_sb"
                                         : "contig_128x128_w4_s2",
                    dg::kContiguous);
  }
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d; p.m_indices = m_indices;
  p.num_groups = num_groups;
  fill_common(p, *c, m, n, k);
  if (int s = set_num_tiles(p, 1)) return s;
  return launch(*c, p, p.num_tiles, (hipStream_t)stream);
}

// Masked-layout tiles (16 experts, max_m 256, N 4096, K 7168, counts uniform
// on 0..c, one process, same inputs; the 256-column tiles of the SwiGLU
// epilogue move the same way):
//  * while every expert fits one 128-row tile, 128 x 256 tiles with three
//    LDS stages stream B fastest: 77-85 us for c = 16-64 (6.1-5.6 TB/s) and
//    108 us for c = 128, against 90-113 us for the 256 x 256 interleaved
//    schedule and 118-124 us for the ping-pong one.  An expert past 128 rows
//    needs a second row of tiles that waits for a free CU (one workgroup per
//    CU): 166-202 us for c = 160-256.
//  * the 256 x 256 interleaved schedule leads up to c = 160 (123 against
//    128 us), the ping-pong one from c = 192 (131-139 against 140-164 us).
//  * a later sweep on the same inputs (counts uniform on 0..c, medians): for
//    c = 128 the 128-row tile takes 104 us against 123 us interleaved and
//    127 us ping-pong; for c = 192 ping-pong 139-141, interleaved 145-148,
//    the 128-row tile 184 us.
// So: max_m <= 128 (no expert can pass 128 rows) or a typical count
// (expected_m) up to 64 picks the 128-row tile when there are enough of its
// tiles to cover half the CUs; a typical count up to 80 the interleaved
// 256 x 256 schedule; larger or unknown (0) counts the ping-pong one.
enum class MaskedTile { kRows128, kInterleaved, kPingPong };
MaskedTile masked_tile(int num_groups, int max_m, int n, int expected_m, const DeviceInfo* info) {
  const bool enough = 2LL * num_groups * ((n + 255) / 256) >= info->cus;
  if (enough && (max_m <= 128 || (expected_m > 0 && expected_m <= 64))) return MaskedTile::kRows128;
  if (expected_m > 0 && expected_m <= 80) return MaskedTile::kInterleaved;
  return MaskedTile::kPingPong;
}

int dg_m_grouped_fp8_gemm_nt_masked(const uint8_t* a, const float* sfa, const uint8_t* b,
                                    const float* sfb, uint16_t* d, const int32_t* masked_m,
                                    int num_groups, int max_m, int n, int k, int expected_m,
                                    dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !d || !masked_m)
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (num_groups < 0) return fail(DG_ERR_INVALID_ARGUMENT, "num_groups must be >= 0 (got %d)", num_groups);
  if (max_m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "max_m must be >= 0 (got %d)", max_m);
  if (expected_m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "expected_m must be >= 0 (got %d)", expected_m);
  if (int s = check_k_n(n, k)) return s;
  if (int s = check_rows(max_m, k)) return s;
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(d) ||
      (reinterpret_cast<uintptr_t>(masked_m) & 3u))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned (masked_m 4-byte)");
  if (num_groups == 0 || max_m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = forced_config(dg::kMasked, &c)) return s;
  if (!c) {
    const MaskedTile t = masked_tile(num_groups, max_m, n, expected_m, info);
    c = find_config(t == MaskedTile::kRows128 ? "masked_128x256_w8_s3"
                    : max_m <= 64             ? "masked_64x64_w4_s3"
                    : t == MaskedTile::kInterleaved ? "masked_256x256_w8_s2"
                                                    : "masked_256x256_w8_s2_pp",
                    dg::kMasked);
  }
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d; p.masked_m = masked_m;
  p.num_groups = num_groups;
  fill_common(p, *c, max_m, n, k);
  if (int s = set_num_tiles(p, num_groups)) return s;
  return launch(*c, p, p.num_tiles, (hipStream_t)stream);
}

int dg_k_grouped_fp8_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d,
                             const int32_t* k_sizes, int num_groups, int m, int n, int k, dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !d || !k_sizes) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (num_groups < 0) return fail(DG_ERR_INVALID_ARGUMENT, "num_groups must be >= 0 (got %d)", num_groups);
  if (int s = check_k_n(n, k)) return s;
  if (int s = check_rows(m, k)) return s;
  if ((long long)num_groups * m * n > 0x7FFFFFFFFFFFLL)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "output too large");
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(d) ||
      (reinterpret_cast<uintptr_t>(k_sizes) & 3u))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned (k_sizes 4-byte)");
  if (m == 0 || num_groups == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = forced_config(dg::kKGrouped, &c)) return s;
  // M up to 2048: the one-B-buffer tile, 507 against 550 us for the 256 x 256
  // tile on 4 x 8192 K, M 2048, N 7168.  At M 4096 the two are level (981
  // against 983 us) and the one-B-buffer tile fetches twice the bytes from
  // beyond L2 (4.0 against 2.0 GB per launch), so 256 x 256 stays.
  if (!c)
    c = find_config(m <= 256 || n <= 256 ? "kgrouped_128x128_w4_s2"
                    : m <= 2048          ? "kgrouped_128x256_w4_s2_sb"
                                         : "kgrouped_256x256_w8_s2",
                    dg::kKGrouped);
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.d = d; p.k_sizes = k_sizes;
  p.num_groups = num_groups;
  fill_common(p, *c, m, n, k);
  if (int s = set_num_tiles(p, num_groups)) return s;
  p.splits = 1;
  p.split_slabs = p.kb_count;
  return launch(*c, p, p.num_tiles, (hipStream_t)stream);
}

int dg_m_grouped_fp8_gemm_nt_masked_swiglu(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                                           uint8_t* hq, float* hs, const int32_t* masked_m, int num_groups,
                                           int max_m, int inter, int k, int expected_m, dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !hq || !hs || !masked_m)
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (num_groups < 0) return fail(DG_ERR_INVALID_ARGUMENT, "num_groups must be >= 0 (got %d)", num_groups);
  if (max_m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "max_m must be >= 0 (got %d)", max_m);
  if (expected_m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "expected_m must be >= 0 (got %d)", expected_m);
  if (inter < 128 || inter % 128 != 0 || inter > (1 << 29))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "inter must be a positive multiple of 128 (got %d)", inter);
  if (int s = check_k_n(2 * inter, k)) return s;
  if (int s = check_rows(max_m, k)) return s;
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(hq) || !aligned16(hs) ||
      (reinterpret_cast<uintptr_t>(masked_m) & 3u))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned (masked_m 4-byte)");
  if (num_groups == 0 || max_m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = forced_config(dg::kMasked, &c, dg::kFp8, dg::kEpiSwigluFp8)) return s;
  if (!c) {
    const MaskedTile t = masked_tile(num_groups, max_m, 2 * inter, expected_m, info);
    c = find_config(t == MaskedTile::kRows128 ? "swiglu_128x256_w8_s3"
                    : max_m <= 64             ? "swiglu_64x256_w4_s3"
                    : t == MaskedTile::kInterleaved ? "swiglu_256x256_w8_s2"
                                                    : "swiglu_256x256_w8_s2_pp",
                    dg::kMasked, dg::kFp8, dg::kEpiSwigluFp8);
  }
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.masked_m = masked_m;
  p.hq = hq; p.hs = hs; p.inter = inter;
  p.num_groups = num_groups;
  fill_common(p, *c, max_m, 2 * inter, k);
  p.tiles_n = inter / 128;  // one tile per 128 h columns (128 gate + 128 up rows of B)
  if (int s = set_num_tiles(p, num_groups)) return s;
  return launch(*c, p, p.num_tiles, (hipStream_t)stream);
}

int dg_m_grouped_fp8_gemm_nt_contiguous_swiglu(const uint8_t* a, const float* sfa, const uint8_t* b,
                                               const float* sfb, uint8_t* hq, float* hs, const int32_t* m_indices,
                                               int m, int inter, int k, int num_groups, dg_stream_t stream) {
  if (!a || !sfa || !b || !sfb || !hq || !hs || !m_indices)
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (num_groups < 1) return fail(DG_ERR_INVALID_ARGUMENT, "num_groups must be >= 1 (got %d)", num_groups);
  if (inter < 128 || inter % 128 != 0 || inter > (1 << 29))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "inter must be a positive multiple of 128 (got %d)", inter);
  if (int s = check_k_n(2 * inter, k)) return s;
  if (m % 128 != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "m must be a multiple of the 128-row alignment (got %d)", m);
  if (int s = check_rows(m, k)) return s;
  if ((long long)m * inter > 0xFFFFFFFFLL) return fail(DG_ERR_UNSUPPORTED_SHAPE, "h must stay below 4 GiB");
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(hq) || !aligned16(hs) ||
      (reinterpret_cast<uintptr_t>(m_indices) & 3u))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned (m_indices 4-byte)");
  if (m == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const Config* c;
  if (int s = forced_config(dg::kContiguous, &c, dg::kFp8, dg::kEpiSwigluFp8)) return s;
  if (!c) {
    // the contiguous GEMM's rule on its 256-column tiles
    const long long tiles = (long long)(m / 128) * (inter / 128);
    const long long t128 = 2 * tiles;
    c = find_config(t128 <= 128        ? "swiglu_contig_64x256_w4_s3"
                    : tiles >= info->cus ? "swiglu_contig_128x256_w4_s2_sb"
                                         : "swiglu_contig_128x256_w8_s3",
                    dg::kContiguous, dg::kFp8, dg::kEpiSwigluFp8);
  }
  dg::GemmParams p{};
  p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.m_indices = m_indices;
  p.hq = hq; p.hs = hs; p.inter = inter;
  p.num_groups = num_groups;
  fill_common(p, *c, m, 2 * inter, k);
  p.tiles_n = inter / 128;  // one tile per 128 h columns (128 gate + 128 up rows of B)
  if (int s = set_num_tiles(p, 1)) return s;
  return launch(*c, p, p.num_tiles, (hipStream_t)stream);
}

int dg_quantize_a_1x128(const float* x, uint8_t* q, float* sfa, int m, int k, dg_stream_t stream) {
  return quantize_a(reinterpret_cast<const void*>(&dg::quant_a_kernel), x, q, sfa, m, k, stream);
}

int dg_quantize_b_128x128(const float* x, uint8_t* q, float* sfb, int n, int k, dg_stream_t stream) {
  return quantize_b(reinterpret_cast<const void*>(&dg::quant_b_kernel), x, q, sfb, n, k, stream);
}

int dg_quantize_a_1x128_fp4(const float* x, uint8_t* q, float* sfa, int m, int k, dg_stream_t stream) {
  return quantize_a(reinterpret_cast<const void*>(&dg::quant_a_fp4_kernel), x, q, sfa, m, k, stream);
}

int dg_quantize_b_128x128_fp4(const float* x, uint8_t* q, float* sfb, int n, int k, dg_stream_t stream) {
  return quantize_b(reinterpret_cast<const void*>(&dg::quant_b_fp4_kernel), x, q, sfb, n, k, stream);
}

int dg_bf16_w4_gemm_nt(const uint16_t* a, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                       uint16_t* d, int m, int n, int k, int group, int format, dg_stream_t stream) {
  if (!codes || !scales || (m > 0 && (!a || !d))) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  if (int s = check_w4(n, k, group, format, zeros)) return s;
  if (!aligned16(a) || !aligned16(codes) || !aligned16(scales) || !aligned16(d) || !aligned16(zeros))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (m == 0) return ok();
  const char* way;
  if (int s = forced_way(kW4RowsName, kW4TileName, &way)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const W4Plan w = w4_plan(m, n, k, group, format, info, way);
  if (w.grid.y > 65535 || w.grid.z > 65535) return fail(DG_ERR_UNSUPPORTED_SHAPE, "m too large (%d)", m);
  const int units = (k + 127) / 128;
  dg::W4Params p{a, codes, scales, zeros, d, m, n, k, nullptr, nullptr, units / (int)w.grid.y, units % (int)w.grid.y};
  if (w.partial_bytes) {
    char* base = nullptr;
    if (int s = ensure_workspace(dev, (hipStream_t)stream, w.partial_bytes, &base)) return s;
    p.count = (int*)base;
    p.partial = (float*)(base + kWsHeader);
  }
  void* args[] = {&p};
  return launch_plain(w.name, w.fn, w.grid, w.threads, args, stream, w.smem, true);
}

int dg_bf16_w4_workspace_size(int m, int n, int k, int group, int format, size_t* bytes) {
  if (!bytes) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  *bytes = 0;
  if (m < 0) return fail(DG_ERR_INVALID_ARGUMENT, "m must be >= 0 (got %d)", m);
  const uint8_t any = 0;
  if (int s = check_w4(n, k, group, format, format == DG_W4_U4 ? &any : nullptr)) return s;
  if (m == 0) return ok();
  const char* way;
  if (int s = forced_way(kW4RowsName, kW4TileName, &way)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  *bytes = w4_plan(m, n, k, group, format, info, way).partial_bytes;
  return ok();
}

int dg_quantize_b_w4(const void* x, int x_bf16, uint8_t* codes, uint16_t* scales, uint8_t* zeros, int n, int k,
                     int group, int format, dg_stream_t stream) {
  if (!x || !codes || !scales) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (int s = check_w4(n, k, group, format, zeros)) return s;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  long long total8 = (long long)n * k / 8;
  const long long blocks = (total8 + 255) / 256;
  if (blocks >= (1LL << 24)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "weight too large (%d x %d)", n, k);
  const void* fn = format == DG_W4_E2M1
                       ? (x_bf16 ? w4_quant_fn<dg::kW4E2m1, true>(group) : w4_quant_fn<dg::kW4E2m1, false>(group))
                       : (x_bf16 ? w4_quant_fn<dg::kW4U4, true>(group) : w4_quant_fn<dg::kW4U4, false>(group));
  void* args[] = {&x, &codes, &scales, &zeros, &total8};
  return launch_plain("w4_quant", fn, dim3((unsigned)blocks), 256, args, stream);
}

int dg_dequantize_b_w4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, uint16_t* w, int n, int k,
                       int group, int format, dg_stream_t stream) {
  if (!codes || !scales || !w) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (int s = check_w4(n, k, group, format, zeros)) return s;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros))
    return fail(DG_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  long long total8 = (long long)n * k / 8;
  const long long blocks = (total8 + 255) / 256;
  if (blocks >= (1LL << 24)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "weight too large (%d x %d)", n, k);
  const void* fn = format == DG_W4_E2M1 ? w4_dequant_fn<dg::kW4E2m1>(group) : w4_dequant_fn<dg::kW4U4>(group);
  void* args[] = {&codes, &scales, &zeros, &w, &total8};
  return launch_plain("w4_dequant", fn, dim3((unsigned)blocks), 256, args, stream);
}

int dg_kv8_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, uint8_t* k_codes,
                  uint8_t* v_codes, float* k_scales, float* v_scales, const int32_t* block_table,
                  const int32_t* ctx_lens, const int32_t* cu_new, int batch, int total, int max_new, int h_kv, int d,
                  int block, int num_blocks, int max_blocks, dg_stream_t stream) {
  if ((batch != 0 && !ctx_lens) || !cu_new || (total > 0 && (!k || !v)))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  dg::Kv8AppendParams p{};
  if (int s = check_cache(k_codes, v_codes, k_scales, v_scales, block_table, batch, h_kv, d, block, num_blocks,
                          max_blocks, &p.c)) return s;
  if (int s = check_batch(batch, total, max_new)) return s;
  if (int s = check_packed(k, k_stride, h_kv, d, "k")) return s;
  if (int s = check_packed(v, v_stride, h_kv, d, "v")) return s;
  if ((reinterpret_cast<uintptr_t>(ctx_lens) & 3u) || (reinterpret_cast<uintptr_t>(cu_new) & 3u))
    return fail(DG_ERR_MISALIGNED, "lengths must be 4-byte aligned");
  if (batch == 0 || total == 0 || max_new == 0 || num_blocks == 0 || max_blocks == 0) return ok();
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.ctx = ctx_lens;
  p.cu = cu_new;
  p.total = total;
  p.most = max_new < total ? max_new : total;
  // blocks that max_new tokens can touch, wherever the first one stands
  const int slots = (p.most + block - 2) / block + 1;
  if ((long long)slots >= (1LL << 24)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many new tokens (%d)", p.most);
  // up to 4 new tokens are at most two groups of 4 positions of a block: one
  // wave holds them (single tokens, 8 heads of 128, one wave / four: 64
  // sequences 6.3 / 6.9 us, 128 in blocks of 16 6.4 / 8.1, one 4.6 / 4.5)
  const bool few = p.most <= 4;
  const int threads = few ? 64 : 256;
  const int items = few ? 1 : (block * d + 8191) / 8192;  // of 4 tokens by 8 values, per thread
  const void* fn = few ? (d == 64    ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<64, 1, 64>)
                          : d == 128 ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<128, 1, 64>)
                                     : reinterpret_cast<const void*>(&dg::kv8_append_kernel<256, 1, 64>))
                   : d == 64 ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<64, 1, 256>)
                   : d == 128 ? (items == 1 ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<128, 1, 256>)
                                            : reinterpret_cast<const void*>(&dg::kv8_append_kernel<128, 2, 256>))
                   : items == 1 ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<256, 1, 256>)
                   : items == 2 ? reinterpret_cast<const void*>(&dg::kv8_append_kernel<256, 2, 256>)
                                : reinterpret_cast<const void*>(&dg::kv8_append_kernel<256, 4, 256>);
  void* args[] = {&p};
  return launch_plain("kv8_append", fn, dim3(slots, 2 * h_kv, batch), threads, args, stream, d * (block + 16));
}

int dg_kv8_attention_workspace_size(int d, size_t* bytes) {
  if (!bytes) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  *bytes = 0;
  if (d != 64 && d != 128 && d != 256)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "head dimension must be 64, 128 or 256 (got %d)", d);
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  *bytes = kv8_part_floats(kv8_workers(info), d) * sizeof(float);
  return ok();
}

int dg_kv8_attention(const uint16_t* q, int64_t q_stride, const uint8_t* k_codes, const uint8_t* v_codes,
                     const float* k_scales, const float* v_scales, const int32_t* block_table,
                     const int32_t* kv_lens, const int32_t* cu_q, uint16_t* out, float* lse, float scale, int causal,
                     int window, int batch, int total, int max_q, int h_q, int h_kv, int d, int block, int num_blocks,
                     int max_blocks, dg_stream_t stream) {
  if ((batch != 0 && !kv_lens) || !cu_q || (total > 0 && (!q || !out)))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  dg::Kv8AttnParams p{};
  if (int s = check_cache(k_codes, v_codes, k_scales, v_scales, block_table, batch, h_kv, d, block, num_blocks,
                          max_blocks, &p.c)) return s;
  if (int s = check_batch(batch, total, max_q)) return s;
  if (h_q < 1 || h_q % h_kv != 0)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "h_q must be a positive multiple of h_kv = %d (got %d)", h_kv, h_q);
  if (!(scale >= 0.f && scale <= 3.4e38f))
    return fail(DG_ERR_INVALID_ARGUMENT, "scale must be finite and >= 0 (got %g)", (double)scale);
  if (window < 0) return fail(DG_ERR_INVALID_ARGUMENT, "window must be >= 0 (got %d)", window);
  if (window > 0 && !causal) return fail(DG_ERR_INVALID_ARGUMENT, "a window goes with causal attention only");
  if (int s = check_packed(q, q_stride, h_q, d, "q")) return s;
  if (!aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(kv_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_q) & 3u))
    return fail(DG_ERR_MISALIGNED, "out must be 16-byte aligned, lse and lengths 4-byte");
  if (batch == 0 || total == 0 || max_q == 0) return ok();
  p.most = max_q < total ? max_q : total;
  if ((long long)p.most * h_q * d > 0x7FFFFFFFLL)  // of one sequence; 32-bit counts of its elements
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many queries per sequence (%d of %d heads)", p.most, h_q);
  const char* way;
  if (int s = forced_way(kKv8Split, kKv8Prompt, &way)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  p.q = q;
  p.q_stride = q_stride;
  p.kv_lens = kv_lens;
  p.cu = cu_q;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.causal = causal != 0;
  p.window = window < (1 << 30) ? window : 1 << 30;  // no sequence is longer: differences stay in 32 bits
  p.batch = batch;
  p.total = total;
  p.h_q = h_q;
  p.group = h_q / h_kv;
  if (num_blocks == 0) p.c.max_blocks = 0;  // no blocks: no tokens, whatever the lengths say
  void* args[] = {&p};
  // Prompts: rows in workgroups of 128 (64 for d = 256) that walk all their
  // keys, if the packed rows fill one for half of the CUs (five eighths for d =
  // 256); else 16-row tiles whose keys are shared out (us, shared out / prompts;
  // 32 / 8 heads of 128: 4 x 256 new of 2048 161 / 69 with 256 such workgroups, 6
  // x 128 of 2048 124 / 66 and 1 x 768 of 4096 169 / 116 with 192, 4 x 128 of 2048
  // 86 / 65, 1 x 512 of 512 35 / 26, 1 x 512 of 4096 112 / 115 and of 16384 382 /
  // 427 with 128, 3 x 128 of 2048 58 / 65 with 96, 1 x 16 of 4096 16 / 109 with 8;
  // 16 / 4 heads of 256: 1 x 640 of 2048 83 / 75 with 160, 4 x 128 of 2048 66 / 75
  // with 128; full tiles are what counts: 16 x 16 of 2048, 16 workgroups of half as
  // many rows a head, 48 / 61).  Sequences of fewer than 64 rows, whose keys a
  // workgroup would walk for them alone, are shared out in a second launch (us,
  // one launch / two: 8 single tokens of 65536 beside a prompt of 2048 1550 / 272,
  // 63 of 32768 1033 / 898, 28 of 8192 beside 4 x 512 of 2048 226 / 193; prompts
  // of unequal lengths pay for it: 4 of up to 2048 behind up to 2048 295 / 303).
  const int prompt_rows = d == 256 ? 64 : 128;
  constexpr int kFew = 64;
  const long long rows = (long long)p.most * p.group, all_rows = (long long)total * p.group;
  const long long prompt_tiles = (rows + prompt_rows - 1) / prompt_rows;
  const long long tiles = min(prompt_tiles * batch, all_rows / prompt_rows);
  bool prompt = rows >= kFew && 8 * tiles * h_kv >= (d == 256 ? 5LL : 4LL) * info->cus, split = true;
  const bool alike = (long long)p.most * batch == total;  // every sequence has max_q rows, if cu is what it should be
  if (prompt && alike) split = false;
  if (way) prompt = way == kKv8Prompt, split = !prompt;
  if (prompt_tiles > 65535) prompt = false, split = true;
  const int border = prompt && split ? kFew : 0;
  char* base = nullptr;
  p.workers = kv8_workers(info);
  if (split)
    if (int s = ensure_workspace(dev, (hipStream_t)stream, kv8_part_floats(p.workers, d) * sizeof(float), &base)) return s;
  if (prompt) {
    p.rows_lo = border;
    p.rows_hi = INT_MAX;
    const void* fn = d == 64    ? reinterpret_cast<const void*>(&dg::kv8_prompt_kernel<64, 2>)
                     : d == 128 ? reinterpret_cast<const void*>(&dg::kv8_prompt_kernel<128, 2>)
                                : reinterpret_cast<const void*>(&dg::kv8_prompt_kernel<256, 1>);
    const int s = launch_plain(kKv8Prompt, fn, dim3(h_kv, batch, (unsigned)prompt_tiles), 256, args, stream);
    if (s || !split) return s;
  }
  p.rows_lo = 0;
  p.rows_hi = border ? border : INT_MAX;
  p.arrived = (int*)base;
  p.part_u = (float*)(base + kWsHeader);
  p.part_ml = p.part_u + (size_t)p.workers * 2 * 16 * d;
  const void* fn = d == 64    ? reinterpret_cast<const void*>(&dg::kv8_attn_kernel<64>)
                   : d == 128 ? reinterpret_cast<const void*>(&dg::kv8_attn_kernel<128>)
                              : reinterpret_cast<const void*>(&dg::kv8_attn_kernel<256>);
  return launch_plain(kKv8Split, fn, dim3(p.workers), 256, args, stream);
}

int dg_latent_append(const uint16_t* latent, int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
                     void* cache_latent, uint16_t* cache_rope, float* cache_scales, const int32_t* block_table,
                     const int32_t* ctx_lens, const int32_t* cu_new, const float* angles, int positions,
                     const uint16_t* norm, float eps, const uint16_t* q, int64_t q_stride, int64_t q_head_stride,
                     uint16_t* q_out, int64_t q_out_stride, int64_t q_out_head_stride, int interleaved, int batch,
                     int total, int max_new, int h_q, int latent_dim, int block, int num_blocks, int max_blocks,
                     dg_stream_t stream) {
  if ((batch != 0 && !ctx_lens) || !cu_new || (total > 0 && (!latent || !rope)) || (positions > 0 && !angles) ||
      (q && !q_out))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  dg::LatentAppendParams p{};
  if (int s = check_latent_cache(cache_latent, cache_rope, cache_scales, block_table, batch, latent_dim, block,
                                 num_blocks, max_blocks, &p.c)) return s;
  if (int s = check_batch(batch, total, max_new)) return s;
  const int rope_dim = latent_dim / 8;
  if (int s = check_packed(latent, latent_stride, 1, latent_dim, "latent")) return s;
  if (int s = check_packed(rope, rope_stride, 1, rope_dim, "rope")) return s;
  if (positions < 0) return fail(DG_ERR_INVALID_ARGUMENT, "positions must be >= 0 (got %d)", positions);
  if (!(eps >= 0.f && eps <= 3.4e38f)) return fail(DG_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0 (got %g)", (double)eps);
  if (q) {
    if (h_q < 1 || h_q > 32767) return fail(DG_ERR_INVALID_ARGUMENT, "h_q must be 1..32767 (got %d)", h_q);
    if (int s = check_strided(q, q_stride, q_head_stride, h_q, rope_dim, 8, "q")) return s;
    if (int s = check_strided(q_out, q_out_stride, q_out_head_stride, h_q, rope_dim, 8, "q_out")) return s;
    if (int s = check_apart(q_out_stride, q_out_head_stride, total, h_q, rope_dim, "q_out")) return s;
    if (q == q_out && (q_stride != q_out_stride || q_head_stride != q_out_head_stride))
      return fail(DG_ERR_INVALID_ARGUMENT, "in place q and q_out must have the same strides");
  }
  if (!aligned16(angles) || !aligned16(norm) || !aligned4(ctx_lens) || !aligned4(cu_new))
    return fail(DG_ERR_MISALIGNED, "angles and norm must be 16-byte aligned, lengths 4-byte");
  if (batch == 0 || total == 0 || max_new == 0 || positions == 0) return ok();
  if (total > (1 << 25)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "at most 2^25 new tokens (got %d)", total);
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  p.latent = latent;
  p.rope = rope;
  p.latent_stride = latent_stride;
  p.rope_stride = rope_stride;
  p.ctx = ctx_lens;
  p.cu = cu_new;
  p.angles = angles;
  p.positions = positions;
  p.norm = norm;
  p.eps = eps;
  p.q = q;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.q_head_stride = q_head_stride;
  p.q_out_stride = q_out_stride;
  p.q_out_head_stride = q_out_head_stride;
  p.h_q = q ? h_q : 0;
  p.batch = batch;
  p.total = total;
  p.most = max_new;
  const bool f8 = cache_scales != nullptr;
  const void* fn = latent_dim == 512 ? latent_append_fn<512>(f8, interleaved != 0) : latent_append_fn<256>(f8, interleaved != 0);
  const int parts = p.h_q > dg::kLatentHeads ? (p.h_q + dg::kLatentHeads - 1) / dg::kLatentHeads : 1;
  void* args[] = {&p};
  return launch_plain("latent_append", fn, dim3((total + 3) / 4, parts), 256, args, stream);
}

int dg_latent_gather(const void* cache_latent, const uint16_t* cache_rope, const float* cache_scales,
                     const int32_t* block_table, const int32_t* starts, const int32_t* cu, uint16_t* latent,
                     uint16_t* rope, int batch, int total, int latent_dim, int block, int num_blocks, int max_blocks,
                     dg_stream_t stream) {
  if (!cu || (total > 0 && (!latent || !rope))) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  dg::LatentGatherParams p{};
  if (int s = check_latent_cache(cache_latent, cache_rope, cache_scales, block_table, batch, latent_dim, block,
                                 num_blocks, max_blocks, &p.c)) return s;
  if (int s = check_batch(batch, total, 0)) return s;
  if (!aligned16(latent) || !aligned16(rope) || !aligned4(starts) || !aligned4(cu))
    return fail(DG_ERR_MISALIGNED, "rows must be 16-byte aligned, lengths 4-byte");
  if (batch == 0 || total == 0 || p.c.max_blocks == 0) return ok();
  if (total > (1 << 25)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "at most 2^25 rows (got %d)", total);
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  p.starts = starts;
  p.cu = cu;
  p.latent = latent;
  p.rope = rope;
  p.batch = batch;
  p.total = total;
  const bool f8 = cache_scales != nullptr;
  const void* fn = latent_dim == 512 ? latent_gather_fn<512>(f8) : latent_gather_fn<256>(f8);
  void* args[] = {&p};
  constexpr int kRows = 4 * dg::kLatentGather;
  return launch_plain("latent_gather", fn, dim3((total + kRows - 1) / kRows), 256, args, stream);
}

int dg_latent_attention_workspace_size(int latent_dim, int max_q, int h_q, size_t* bytes) {
  if (!bytes) return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  *bytes = 0;
  if (int s = check_latent_dim(latent_dim)) return s;
  if (max_q < 0) return fail(DG_ERR_INVALID_ARGUMENT, "max_q must be >= 0 (got %d)", max_q);
  if (int s = check_latent_rows(max_q, h_q)) return s;
  const char* forced;
  if (int s = forced_name(&forced)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  const int tiles = latent_row_tiles(max_q, h_q, LLONG_MAX / 4096, info->cus, forced);  // the most that any tokens take
  *bytes = latent_part_bytes(info->cus, tiles, latent_dim);
  return ok();
}

int dg_latent_attention(const uint16_t* q, int64_t q_stride, int64_t q_head_stride, const uint16_t* q_rope,
                        int64_t q_rope_stride, int64_t q_rope_head_stride, const void* cache_latent,
                        const uint16_t* cache_rope, const float* cache_scales, const int32_t* block_table,
                        const int32_t* kv_lens, const int32_t* cu_q, uint16_t* out, int64_t out_stride,
                        int64_t out_head_stride, float* lse, float scale, int causal, int batch, int total, int max_q,
                        int h_q, int latent_dim, int block, int num_blocks, int max_blocks, dg_stream_t stream) {
  if ((batch != 0 && !kv_lens) || !cu_q || (total > 0 && (!q || !q_rope || !out)))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  dg::LatentAttnParams p{};
  if (int s = check_latent_cache(cache_latent, cache_rope, cache_scales, block_table, batch, latent_dim, block,
                                 num_blocks, max_blocks, &p.c)) return s;
  if (int s = check_batch(batch, total, max_q)) return s;
  if (int s = check_latent_rows(max_q, h_q)) return s;
  if (!(scale >= 0.f && scale <= 3.4e38f))
    return fail(DG_ERR_INVALID_ARGUMENT, "scale must be finite and >= 0 (got %g)", (double)scale);
  if (int s = check_strided(q, q_stride, q_head_stride, h_q, latent_dim, 8, "q")) return s;
  if (int s = check_strided(q_rope, q_rope_stride, q_rope_head_stride, h_q, latent_dim / 8, 8, "q_rope")) return s;
  if (int s = check_strided(out, out_stride, out_head_stride, h_q, latent_dim, 8, "out")) return s;
  if (int s = check_apart(out_stride, out_head_stride, total, h_q, latent_dim, "out")) return s;
  if (!aligned4(lse) || !aligned4(kv_lens) || !aligned4(cu_q))
    return fail(DG_ERR_MISALIGNED, "lse and lengths must be 4-byte aligned");
  if (batch == 0 || total == 0 || max_q == 0) return ok();
  const char* forced;
  if (int s = forced_name(&forced)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  if (int s = ensure_latent_attributes(dev)) return s;
  p.q = q;
  p.qr = q_rope;
  p.q_stride = q_stride;
  p.q_head_stride = q_head_stride;
  p.qr_stride = q_rope_stride;
  p.qr_head_stride = q_rope_head_stride;
  p.kv_lens = kv_lens;
  p.cu = cu_q;
  p.out = out;
  p.out_stride = out_stride;
  p.out_head_stride = out_head_stride;
  p.lse = lse;
  p.scale_log2 = latent_scale(scale);
  p.causal = causal != 0;
  p.batch = batch;
  p.total = total;
  p.most = max_q;
  p.h_q = h_q;
  p.workers = info->cus;
  const long long all_blocks = (long long)batch * max_blocks;
  const long long tokens = (all_blocks < num_blocks ? all_blocks : num_blocks) * block;
  const int tiles = latent_row_tiles(max_q, h_q, tokens, p.workers, forced);
  const LatentKernel k = latent_attn(latent_dim, cache_scales != nullptr, tiles);
  const int row_tiles = (int)(((long long)max_q * h_q + 16 * tiles - 1) / (16 * tiles));
  p.together = (long long)max_q * batch == total && row_tiles <= 8 ? row_tiles : 1;
  char* base = nullptr;
  if (int s = ensure_workspace(dev, (hipStream_t)stream, latent_part_bytes(p.workers, tiles, latent_dim), &base)) return s;
  p.part_u = (float*)(base + kWsHeader);
  p.part_ml = p.part_u + (size_t)p.workers * 2 * 16 * tiles * latent_dim;
  p.cut = (dg::LatentCut*)(p.part_ml + (size_t)p.workers * 2 * 16 * tiles * 2);
  void* args[] = {&p};
  if (int s = launch_plain("latent_attention", k.fn, dim3(p.workers), 256, args, stream, k.smem)) return s;
  return launch_plain("latent_join", k.join, dim3(4 * p.workers), 256, args, stream);
}

int dg_latent_expanded_attention(const uint16_t* q, int64_t q_stride, const uint16_t* kv, int64_t kv_stride,
                                 const uint16_t* k_rope, int64_t k_rope_stride, const int32_t* cu_q,
                                 const int32_t* cu_kv, uint16_t* out, float* lse, float scale, int causal, int batch,
                                 int total, int total_kv, int max_q, int heads, int head_dim, dg_stream_t stream) {
  if (!cu_q || !cu_kv || (total > 0 && (!q || !out)) || (total_kv > 0 && (!kv || !k_rope)))
    return fail(DG_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (head_dim != 64 && head_dim != 128)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64 or 128 (got %d)", head_dim);
  if (heads < 1 || heads > 32767) return fail(DG_ERR_INVALID_ARGUMENT, "heads must be 1..32767 (got %d)", heads);
  if (int s = check_batch(batch, total, max_q)) return s;
  if (total_kv < 0) return fail(DG_ERR_INVALID_ARGUMENT, "token counts must be >= 0");
  if (!(scale >= 0.f && scale <= 3.4e38f))
    return fail(DG_ERR_INVALID_ARGUMENT, "scale must be finite and >= 0 (got %g)", (double)scale);
  if (int s = check_packed(q, q_stride, heads, head_dim / 2 * 3, "q")) return s;
  if (int s = check_packed(kv, kv_stride, heads, 2 * head_dim, "kv")) return s;
  if (int s = check_packed(k_rope, k_rope_stride, 1, head_dim / 2, "k_rope")) return s;
  if (kv_stride >= (1 << 26) || k_rope_stride >= (1 << 26))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "kv and k_rope: strides must stay below 2^26 elements");
  if (!aligned16(out) || !aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_kv))
    return fail(DG_ERR_MISALIGNED, "out must be 16-byte aligned, lse and lengths 4-byte");
  if (batch == 0 || total == 0 || max_q == 0) return ok();
  const char* forced;
  if (int s = forced_name(&forced)) return s;
  int dev;
  DeviceInfo* info;
  if (int s = current_device(&dev, &info)) return s;
  if (int s = ensure_latent_attributes(dev)) return s;
  dg::LatentExpandedParams p{};
  p.q = q;
  p.kv = kv;
  p.kr = k_rope;
  p.q_stride = q_stride;
  p.kv_stride = kv_stride;
  p.kr_stride = k_rope_stride;
  p.cu = cu_q;
  p.cu_kv = cu_kv;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = latent_scale(scale);
  p.causal = causal != 0;
  p.batch = batch;
  p.total = total;
  p.total_kv = total_kv;
  p.most = max_q < total ? max_q : total;
  p.h = heads;
  // Queries of a head that a workgroup takes: 128, or 64 where there would be no
  // more workgroups of 128 than CUs or none would be more than half full, as a
  // step then takes a workgroup, alone on its CU, less; and 32 or 16, with the
  // tokens shared out between the waves, where all workgroups of that many are
  // resident at once, one a CU (heads of 128) or two (of 64): the way through the
  // tokens is a quarter as long, but each workgroup fetches all of them again.
  // us with 16 / 32 / 64 / 128 queries, heads of 128:
  //   32 heads, 1 x 128 new of 2048    27 / 35 / 49 / 67     8 heads, 1 x 4 of 8192     77 / 107 / 166 / 224
  //   16 heads, 8 x 20 of up to 4096   62 / 74 / 115 / 144   24 heads, 1 x 256 of 2048  45 / 35 / 50 / 69
  //   40 heads, 1 x 128 of 2048        50 / 36 / 51 / 71     36 heads, 1 x 256 of 2048  72 / 64 / 51 / 70
  //   32 heads, 1 x 512 of 2048        91 / 65 / 53 / 70     32 heads, 1 x 1024         85 / 59 / 34 / 44
  //   32 heads, 4 x 512 of 2048       372 / 246 / 125 / 99   16 heads, 30 x 8 of 500    24 / 29 / 24 / 28
  // heads of 64:
  //   5 heads, 9 x up to 150           7.0 / 7.7 / 8.9 / 10  16 heads, 1 x 512 of 4096  39 / 39 / 64 / 83
  //   32 heads, 1 x 512 of 1024        23 / 16 / 19 / 25     32 heads, 4 x up to 1024 of 2048  186 / 99 / 60 / 62
  const auto tiles_of = [&](int rows) { return ((long long)p.most + rows - 1) / rows; };
  const auto groups = [&](int rows) {  // at most, whatever the lengths
    const long long by_longest = tiles_of(rows) * batch, by_total = total / rows + batch;
    return heads * (by_longest < by_total ? by_longest : by_total);
  };
  const int resident = head_dim == 128 ? info->cus : 2 * info->cus;
  int rows = groups(16) <= resident ? 16 : groups(32) <= resident ? 32 : groups(128) <= info->cus || p.most <= 64 ? 64 : 128;
  for (int i = 0; forced && i < 4; ++i)
    if (strcmp(forced, kLatentPrompt[i]) == 0) rows = 16 << i;
  const long long tiles = tiles_of(rows);
  if (tiles > 65535) return fail(DG_ERR_UNSUPPORTED_SHAPE, "too many queries per sequence (%d)", p.most);
  const LatentKernel k = latent_expanded(head_dim, rows);
  void* args[] = {&p};
  return launch_plain("latent_expanded_attention", k.fn, dim3(heads, batch, (unsigned)tiles), 256, args, stream, k.smem);
}

}  // extern "C"
