// Runs the library's host code on a machine without a GPU and looks at every
// kernel launch it makes: the sources are compiled for the host alone against
// the stand-in HIP runtime below, whose hipLaunchKernel inspects the launch
// instead of running it. Built and run by tests/test_launch_parameters.py
// with uninitialised variables filled with the byte 0xAA, so that a field of a
// kernel's parameters that nobody set shows as that pattern.
//
// Checked for every launch: the parameters hold no unset 8-byte word and a
// packed base with the fields its operator stands for (half and half_s2 zero
// unless it is the joint base of two projections), and grid, block and LDS are
// within the device's limits. Prints the number of launches of every kernel
// and "ok".
#include <cstring>
#include <limits>
#include <string>

#include "lora4.hip"

#define VISIBLE extern "C" __attribute__((visibility("default")))

// the device code that is not there
asm(".data\n.globl __hip_fatbin\n.p2align 12\n__hip_fatbin:\n.quad 0\n.text\n");

namespace {

int failures = 0;

void fail(const char *what, const char *detail) {
  std::printf("FAIL %s: %s\n", what, detail);
  ++failures;
}

std::map<const void *, std::string> &kernels() {
  static std::map<const void *, std::string> k;
  return k;
}
std::map<std::string, int> counts;

struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t st;
} pushed;

std::string context;      // the call under way
bool joint = false;       // its dX runs over the joint base of two projections
int64_t joint_half = 0;

bool is(const std::string &name, const char *kernel) {   // (mangled: <length><name>)
  return name.find(std::to_string(std::strlen(kernel)) + kernel) != std::string::npos;
}

// An 8-byte word of fields is never 0xAAAA... by intent, and padding is
// shorter than 8 bytes.
template <typename T>
const T &checked(const std::string &name, const void *arg) {
  const unsigned char *b = reinterpret_cast<const unsigned char *>(arg);
  for (size_t i = 0; i + 8 <= sizeof(T); i += 8) {
    uint64_t w;
    std::memcpy(&w, b + i, 8);
    if (w == 0xAAAAAAAAAAAAAAAAull)
      fail(context.c_str(), (name + ": unset word at byte " + std::to_string(i)).c_str());
  }
  return *reinterpret_cast<const T *>(arg);
}

void check_base(const std::string &name, const lora4::PackedW &w, bool dgrad) {
  const bool two = dgrad && joint;
  if (w.half != (two ? joint_half : 0)) fail(context.c_str(), (name + ": half " + std::to_string(w.half)).c_str());
  if (w.half_s2 != (two && w.scales2 ? w.g_scales2 / 2 : 0))
    fail(context.c_str(), (name + ": half_s2 " + std::to_string(w.half_s2)).c_str());
  if (w.shared != 0 && w.shared != 1) fail(context.c_str(), (name + ": shared").c_str());
}

void inspect(const std::string &name, void **args) {
  if (is(name, "k_gemm_nt")) check_base(name, checked<lora4::NtParams>(name, args[0]).W, false);
  else if (is(name, "k_gemm_nn")) check_base(name, checked<lora4::NnParams>(name, args[0]).W, true);
  else if (is(name, "k_gemm_tn2")) {
    for (int i = 0; i < 2; ++i) {
      const lora4::TnParams &p = checked<lora4::TnParams>(name, args[i]);
      if (p.half_shift != (joint ? 1 : 0) || (!joint && (p.u_half || p.v_half))) fail(context.c_str(), name.c_str());
    }
  } else if (is(name, "k_gemm_dgrad")) check_base(name, checked<lora4::big::Params>(name, args[0]).W, true);
  else if (is(name, "k_gemm_fwd") || is(name, "k_gemm_fwd_small") || is(name, "k_gemm_fwd_epi") ||
           is(name, "k_gemm_fwd_split") || is(name, "k_gemm_fwd_mx") || is(name, "k_epi_reduce") ||
           is(name, "k_reduce_tiles"))
    check_base(name, checked<lora4::big::Params>(name, args[0]).W, false);
  else if (is(name, "k_small")) check_base(name, checked<lora4::small::Params>(name, args[0]).W, false);
  else if (is(name, "k_small_z")) checked<lora4::small::ZParams>(name, args[0]);
  else if (is(name, "k_act_dz")) checked<lora4::actbwd::DzParams>(name, args[0]);
  else if (is(name, "k_col_part")) checked<lora4::actbwd::ColParams>(name, args[0]);
  else if (is(name, "k_rmsnorm_fwd")) checked<lora4::norm::FwdParams>(name, args[0]);
  else if (is(name, "k_rmsnorm_bwd")) checked<lora4::norm::BwdParams>(name, args[0]);
  else if (is(name, "k_rows_lds") || is(name, "k_rows_skinny")) checked<lora4::skinny::Params>(name, args[0]);
  else {   // (scalars only)
    for (const char *k : {"k_fill_u16", "k_reduce_bf16", "k_col_sum", "k_col_sum_slots", "k_quant_mxfp8"})
      if (is(name, k)) return;
    fail("a kernel this driver does not know", name.c_str());
  }
}

}  // namespace

VISIBLE void **__hipRegisterFatBinary(const void *) {
  static void *handle = nullptr;
  return &handle;
}
VISIBLE void __hipUnregisterFatBinary(void **) {}
VISIBLE void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *, void *, void *,
                                   void *, int *) {
  kernels()[host] = name;
}
VISIBLE void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
VISIBLE hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t st) {
  pushed = {grid, block, lds, st};
  return hipSuccess;
}
VISIBLE hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *st) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *st = pushed.st;
  return hipSuccess;
}
VISIBLE hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t lds, hipStream_t) {
  const auto it = kernels().find(fn);
  if (it == kernels().end()) {
    fail(context.c_str(), "launch of something that is no kernel");
    return hipSuccess;
  }
  const std::string &name = it->second;
  ++counts[name.substr(0, name.find("IL"))];
  if (!grid.x || !grid.y || !grid.z || grid.x > 0x7FFFFFFFu || grid.y > 65535 || grid.z > 65535 ||
      block.x * block.y * block.z > 1024 || (uint64_t)grid.x * block.x > 0xFFFFFFFFull || lds > 160 * 1024)
    fail(context.c_str(), (name + ": launch shape").c_str());
  inspect(name, args);
  return hipSuccess;
}
VISIBLE hipError_t hipGetDevice(int *d) {
  *d = 0;
  return hipSuccess;
}
VISIBLE hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
VISIBLE hipError_t hipFuncSetAttribute(const void *, hipFuncAttribute, int) { return hipSuccess; }
VISIBLE hipError_t hipGetLastError(void) { return hipSuccess; }
VISIBLE hipError_t hipPeekAtLastError(void) { return hipSuccess; }
VISIBLE hipError_t hipGetSymbolAddress(void **p, const void *) {
  *p = reinterpret_cast<void *>((uintptr_t)0x40000000);
  return hipSuccess;
}
VISIBLE hipError_t hipEventCreate(hipEvent_t *) { return hipErrorNotSupported; }
VISIBLE hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipErrorNotSupported; }
VISIBLE hipError_t hipEventSynchronize(hipEvent_t) { return hipErrorNotSupported; }
VISIBLE hipError_t hipEventElapsedTime(float *, hipEvent_t, hipEvent_t) { return hipErrorNotSupported; }
VISIBLE hipError_t hipMemcpyAsync(void *, const void *, size_t, hipMemcpyKind, hipStream_t) {
  return hipErrorNotSupported;
}
VISIBLE hipError_t hipStreamSynchronize(hipStream_t) { return hipErrorNotSupported; }

namespace {

// device addresses: the host code never dereferences them
uint16_t *const D = reinterpret_cast<uint16_t *>((uintptr_t)0x100000);
const int64_t *const OFFS = reinterpret_cast<const int64_t *>((uintptr_t)0x200000);
void *const WS = reinterpret_cast<void *>((uintptr_t)0x10000000);

lora4_W base(int fmt, int64_t N, int64_t K, int64_t groups) {
  const int block = fmt == LORA4_MXFP4 ? 32 : fmt == LORA4_NVFP4 ? 16 : 64;
  return lora4_W{fmt, block, N, K, groups, reinterpret_cast<const uint8_t *>(D), D,
                 fmt == LORA4_NF4_DQ ? reinterpret_cast<const float *>(D) : nullptr};
}

void expect(long got, long want) {
  if (got != want) fail(context.c_str(), ("status " + std::to_string(got) + ", want " + std::to_string(want)).c_str());
}

// A call with the workspace that its size query names.
template <typename Call>
void run(const char *what, const lora4_W &W, int64_t M, int r, size_t bytes, Call &&call) {
  context = std::string(what) + " format " + std::to_string(W.format) + " N " + std::to_string(W.N) + " K " +
            std::to_string(W.K) + " groups " + std::to_string(W.groups) + " M " + std::to_string(M) + " r " +
            std::to_string(r);
  if (!bytes) {
    fail(context.c_str(), "no workspace size");
    return;
  }
  expect(call(bytes), LORA4_OK);
}

void layer(int fmt, int64_t N, int64_t K, int64_t E, int64_t M, int r) {
  const lora4_W W = base(fmt, N, K, E);
  const int64_t *offs = E > 1 ? OFFS : nullptr;
  run("forward", W, M, r, lora4_workspace_bytes(0, &W, M, r), [&](size_t n) {
    return lora4_forward(&W, D, M, D, D, r, 2.0f, offs, D, D, D, D, WS, n, nullptr);
  });
  run("backward", W, M, r, lora4_workspace_bytes(1, &W, M, r), [&](size_t n) {
    return lora4_backward(&W, D, D, M, D, D, r, 2.0f, offs, nullptr, D, D, D, WS, n, nullptr);
  });
  if (M <= 64)
    run("forward_noalloc", W, M, r, 1, [&](size_t) {
      return lora4_forward_noalloc(&W, D, M, D, D, r, 2.0f, offs, D, D, nullptr, nullptr, nullptr);
    });
  if (E > 1) return;
  const int64_t adapters = 5;
  run("forward_multi", W, M, r, lora4_workspace_bytes_multi(0, &W, adapters, M, r), [&](size_t n) {
    return lora4_forward_multi(&W, adapters, D, M, D, D, r, 2.0f, OFFS, D, D, nullptr, nullptr, WS, n, nullptr);
  });
  run("backward_multi", W, M, r, lora4_workspace_bytes_multi(1, &W, adapters, M, r), [&](size_t n) {
    return lora4_backward_multi(&W, adapters, D, D, M, D, D, r, 2.0f, OFFS, D, D, D, D, WS, n, nullptr);
  });
  if (fmt == LORA4_MXFP4)
    run("forward_mx", W, M, r, lora4_workspace_bytes_mx(&W, M, r),
        [&](size_t n) { return lora4_forward_mx(&W, D, M, D, D, r, 2.0f, D, D, WS, n, nullptr); });
}

void feed_forward(int fmt, int64_t N, int64_t K, int64_t E, int64_t M, int r) {
  const int64_t *offs = E > 1 ? OFFS : nullptr;
  const lora4_W G = base(fmt, N, K, 2 * E), W = base(fmt, N, K, E);
  if (r <= 128) {
    run("gated_forward", G, M, r, lora4_gated_workspace_bytes(0, &G, M, r), [&](size_t n) {
      expect(lora4_gated_forward(&G, LORA4_ACT_SILU, D, M, D, D, r, 2.0f, offs, D, D, D, WS, n - 1, nullptr),
             LORA4_ERR_WORKSPACE);
      return lora4_gated_forward(&G, LORA4_ACT_SILU, D, M, D, D, r, 2.0f, offs, D, D, D, WS, n, nullptr);
    });
    joint = true;
    joint_half = lora4::w_blocks(N) * 64;
    for (const uint16_t *Z : {(const uint16_t *)D, (const uint16_t *)nullptr})
      run("gated_backward", G, M, r, lora4_gated_workspace_bytes(1, &G, M, r), [&](size_t n) {
        expect(lora4_gated_backward(&G, LORA4_ACT_GELU, D, D, D, M, D, D, r, 2.0f, offs, Z, D, D, D, WS, n - 1,
                                    nullptr),
               LORA4_ERR_WORKSPACE);
        return lora4_gated_backward(&G, LORA4_ACT_GELU, D, D, D, M, D, D, r, 2.0f, offs, Z, D, D, D, WS, n, nullptr);
      });
    joint = false;
  }
  for (int act : {LORA4_ACT_NONE, LORA4_ACT_GELU_TANH}) {
    run("forward_epilogue", W, M, r, lora4_epilogue_workspace_bytes(0, &W, M, r), [&](size_t n) {
      expect(lora4_forward_epilogue(&W, act, D, M, D, D, r, 2.0f, offs, D, D, D, D, D, WS, n - 1, nullptr),
             LORA4_ERR_WORKSPACE);
      return lora4_forward_epilogue(&W, act, D, M, D, D, r, 2.0f, offs, D, D, D, D, D, WS, n, nullptr);
    });
    for (uint16_t *db : {D, (uint16_t *)nullptr})
      run("backward_epilogue", W, M, r, lora4_epilogue_workspace_bytes(1, &W, M, r), [&](size_t n) {
        return lora4_backward_epilogue(&W, act, D, D, D, M, D, D, r, 2.0f, offs, nullptr, D, D, D, db, WS, n, nullptr);
      });
  }
}

void norms() {
  for (int64_t M : {0, 1, 5, 2100, 70000})
    for (int64_t Dn : {1, 7, 96, 1024, 1025, 5003, 8200, 16375, 16384}) {
      const lora4_W none = base(LORA4_NF4, 1, Dn, 1);
      const bool mx = Dn % 32 == 0;
      uint8_t *u8 = reinterpret_cast<uint8_t *>(D);
      run("rmsnorm", none, M, 0, lora4_rmsnorm_workspace_bytes(M, Dn), [&](size_t n) {
        expect(lora4_rmsnorm_forward(D, D, D, M, Dn, 1e-5f, D, D, mx ? u8 : nullptr, mx ? u8 : nullptr, nullptr),
               LORA4_OK);
        expect(lora4_rmsnorm_backward(D, D, D, D, M, Dn, 1e-5f, D, nullptr, nullptr, 0, nullptr), LORA4_OK);
        expect(lora4_rmsnorm_backward(D, D, D, D, M, Dn, 1e-5f, D, D, WS, n - 1, nullptr),
               M ? LORA4_ERR_WORKSPACE : LORA4_OK);
        return lora4_rmsnorm_backward(D, D, D, D, M, Dn, 1e-5f, D, D, WS, n, nullptr);
      });
    }
  for (int64_t Dn : {0, 16377, 16385}) expect((long)lora4_rmsnorm_workspace_bytes(8, Dn), 0);
}

// Refused arguments of the feed-forward operators (tests/abi_driver.c has the
// others'): one thing wrong at a time, and the status that names it.
void refusals() {
  uint16_t *const MIS = D + 4;   // 8-byte aligned
  uint8_t *const u8 = reinterpret_cast<uint8_t *>(D);
  const size_t n = (size_t)1 << 40;
  const float inf = std::numeric_limits<float>::infinity();
  context = "refusals of the norm";
  auto norm = [&](uint16_t *X, uint16_t *R, uint16_t *w, int64_t M, int64_t Dn, float eps, uint16_t *H, uint16_t *Y,
                  uint8_t *c, uint8_t *sc) {
    return lora4_rmsnorm_forward(X, R, w, M, Dn, eps, H, Y, c, sc, nullptr);
  };
  expect(norm(D, D, D, -1, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, ((int64_t)1 << 31) + 1, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, 4, 0, 1e-5f, D, D, nullptr, nullptr), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, 4, 16385, 1e-5f, D, D, nullptr, nullptr), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, 4, 40, 1e-5f, D, D, u8, u8), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, 4, 256, -1e-5f, D, D, u8, u8), LORA4_ERR_SHAPE);
  expect(norm(D, D, D, 4, 256, inf, D, D, u8, u8), LORA4_ERR_SHAPE);
  expect(norm(nullptr, D, D, 4, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_NULL);
  expect(norm(D, nullptr, D, 4, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_NULL);
  expect(norm(D, D, nullptr, 4, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_NULL);
  expect(norm(D, D, D, 4, 256, 1e-5f, D, nullptr, nullptr, nullptr), LORA4_ERR_NULL);
  expect(norm(D, D, D, 4, 256, 1e-5f, D, D, u8, nullptr), LORA4_ERR_NULL);
  expect(norm(D, MIS, D, 4, 256, 1e-5f, D, D, u8, u8), LORA4_ERR_ALIGN);
  auto norm_bwd = [&](uint16_t *dY, uint16_t *H, uint16_t *w, uint16_t *dX, uint16_t *dW, void *ws, size_t b) {
    return lora4_rmsnorm_backward(dY, H, w, D, 4, 256, 1e-5f, dX, dW, ws, b, nullptr);
  };
  expect(norm_bwd(nullptr, D, D, D, D, WS, n), LORA4_ERR_NULL);
  expect(norm_bwd(D, nullptr, D, D, D, WS, n), LORA4_ERR_NULL);
  expect(norm_bwd(D, D, nullptr, D, D, WS, n), LORA4_ERR_NULL);
  expect(norm_bwd(D, D, D, nullptr, D, WS, n), LORA4_ERR_NULL);
  expect(norm_bwd(D, D, D, MIS, D, WS, n), LORA4_ERR_ALIGN);
  expect(norm_bwd(D, D, D, D, D, nullptr, n), LORA4_ERR_WORKSPACE);
  expect((long)lora4_rmsnorm_workspace_bytes(-1, 8), 0);

  context = "refusals of the gated projections";
  lora4_W G = base(LORA4_NF4, 1000, 512, 2);
  auto gated = [&](const lora4_W *W, int act, uint16_t *X, int64_t M, uint16_t *A, int r, float s, const int64_t *offs,
                   uint16_t *H, void *ws, size_t b) {
    return lora4_gated_forward(W, act, X, M, A, D, r, s, offs, H, D, D, ws, b, nullptr);
  };
  auto gated_bwd = [&](const lora4_W *W, int act, uint16_t *X, int64_t M, uint16_t *A, int r, float s,
                       const int64_t *offs, uint16_t *dH, void *ws, size_t b) {
    return lora4_gated_backward(W, act, X, dH, D, M, A, D, r, s, offs, D, D, D, D, ws, b, nullptr);
  };
  auto both = [&](auto &&call) {
    expect(call(nullptr, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_NULL);
    expect(call(&G, 4, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_FORMAT);
    expect(call(&G, -1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_FORMAT);
    expect(call(&G, 1, D, -1, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    expect(call(&G, 1, D, 16, D, 0, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    expect(call(&G, 1, D, 16, D, 129, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    expect(call(&G, 1, D, 16, D, 16, inf, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    expect(call(&G, 1, D, 16, D, 16, 1.0f, OFFS, D, WS, n), LORA4_ERR_SHAPE);
    expect(call(&G, 1, nullptr, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_NULL);
    expect(call(&G, 1, D, 16, nullptr, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_NULL);
    expect(call(&G, 1, D, 16, D, 16, 1.0f, nullptr, nullptr, WS, n), LORA4_ERR_NULL);
    expect(call(&G, 1, D, 16, MIS, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_ALIGN);
    expect(call(&G, 1, D, 16, D, 16, 1.0f, nullptr, D, nullptr, n), LORA4_ERR_WORKSPACE);
    expect(call(&G, 1, D, 16, D, 16, 1.0f, nullptr, D, MIS, n), LORA4_ERR_ALIGN);
    lora4_W bad = G;
    bad.groups = 3;
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    bad.groups = 4;
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_NULL);
    bad.groups = 0;
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    bad = G;
    bad.format = 9;
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_FORMAT);
    bad = base(LORA4_NF4, (int64_t)1 << 26, 64, 2);   // 2 GiB of codes a group
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_SHAPE);
    bad = base(LORA4_NF4_DQ, 1000, 512, 2);
    bad.scales2 = nullptr;
    expect(call(&bad, 1, D, 16, D, 16, 1.0f, nullptr, D, WS, n), LORA4_ERR_NULL);
  };
  both(gated);
  both(gated_bwd);
  expect((long)lora4_gated_workspace_bytes(2, &G, 16, 16), 0);
  expect((long)lora4_gated_workspace_bytes(0, nullptr, 16, 16), 0);
  expect((long)lora4_gated_workspace_bytes(1, &G, 16, 129), 0);

  context = "refusals of the linear with an epilogue";
  lora4_W W = base(LORA4_NVFP4, 1000, 512, 1);
  auto fwd = [&](int act, int64_t M, int r, const int64_t *offs, uint16_t *bias, uint16_t *R, uint16_t *Y, void *ws,
                 size_t b) {
    return lora4_forward_epilogue(&W, act, D, M, D, D, r, 1.0f, offs, bias, R, Y, D, D, ws, b, nullptr);
  };
  expect(fwd(7, 16, 16, nullptr, D, D, D, WS, n), LORA4_ERR_FORMAT);
  expect(fwd(2, 16, 257, nullptr, D, D, D, WS, n), LORA4_ERR_SHAPE);
  expect(fwd(2, -1, 16, nullptr, D, D, D, WS, n), LORA4_ERR_SHAPE);
  expect(fwd(2, 16, 16, OFFS, D, D, D, WS, n), LORA4_ERR_SHAPE);
  expect(fwd(2, 16, 16, nullptr, MIS, D, D, WS, n), LORA4_ERR_ALIGN);
  expect(fwd(2, 16, 16, nullptr, D, MIS, D, WS, n), LORA4_ERR_ALIGN);
  expect(fwd(2, 16, 16, nullptr, D, D, nullptr, WS, n), LORA4_ERR_NULL);
  expect(fwd(2, 16, 16, nullptr, D, D, D, WS, 16), LORA4_ERR_WORKSPACE);
  auto bwd = [&](int act, uint16_t *P, uint16_t *dA, uint16_t *db, void *ws, size_t b) {
    return lora4_backward_epilogue(&W, act, D, D, P, 16, D, D, 16, 1.0f, nullptr, nullptr, D, dA, D, db, ws, b,
                                   nullptr);
  };
  for (int act : {LORA4_ACT_NONE, LORA4_ACT_SILU}) {
    expect(bwd(act, D, nullptr, D, WS, n), LORA4_ERR_NULL);
    expect(bwd(act, D, D, MIS, WS, n), LORA4_ERR_ALIGN);
    expect(bwd(act, D, D, D, nullptr, n), LORA4_ERR_WORKSPACE);
    expect(bwd(act, D, D, D, WS, 16), LORA4_ERR_WORKSPACE);
    expect(bwd(act, D, D, D, MIS, n), LORA4_ERR_ALIGN);
  }
  expect(bwd(LORA4_ACT_SILU, nullptr, D, D, WS, n), LORA4_ERR_NULL);
  expect(bwd(9, D, D, D, WS, n), LORA4_ERR_FORMAT);
  expect((long)lora4_epilogue_workspace_bytes(0, nullptr, 16, 16), 0);
  expect((long)lora4_epilogue_workspace_bytes(-1, &W, 16, 16), 0);
  expect((long)lora4_epilogue_workspace_bytes(0, &W, 16, 257), 0);
}

// Size queries over the ends of their ranges (no call: nothing that large
// exists), where an overflow of the planning's arithmetic would show.
void sizes() {
  for (int fmt = LORA4_NF4; fmt <= LORA4_NVFP4; ++fmt)
    for (int64_t M : {(int64_t)0, (int64_t)1, (int64_t)3, (int64_t)65537, (int64_t)1 << 24, (int64_t)1 << 31})
      for (int64_t N : {1, 63, 14336, 1 << 20})
        for (int64_t K : {64, 4096, 1 << 17})
          for (int64_t groups : {1, 2, 90, 65534}) {
            const lora4_W W = base(fmt, N, K, groups);
            // (the documented limit: 32-bit offsets within a group's base)
            const int64_t tiles = (N + 63) / 64 * (K / 64);
            if (tiles * 2048 + 4 * (K / 64) * 2048 >= (int64_t)1 << 31) continue;
            context = "sizes M " + std::to_string(M) + " N " + std::to_string(N) + " K " + std::to_string(K) +
                      " groups " + std::to_string(groups);
            for (int r : {1, 128, 256})
              for (int which = 0; which < 2; ++which) {
                if (!lora4_epilogue_workspace_bytes(which, &W, M, r)) fail(context.c_str(), "epilogue size");
                const bool gated = groups % 2 == 0 && r <= 128;
                if ((lora4_gated_workspace_bytes(which, &W, M, r) != 0) != gated) fail(context.c_str(), "gated size");
              }
          }
}

}  // namespace

int main() {
  struct Shape {
    int64_t N, K, E, M;
    int r;
  };
  const Shape shapes[] = {
      {96, 256, 1, 1, 16},      {515, 192, 1, 300, 128},  {14336, 4096, 1, 8, 16},   {14336, 4096, 1, 24, 64},
      {4096, 14336, 1, 16, 16}, {4096, 4096, 1, 333, 24}, {4096, 4096, 1, 2048, 32}, {14336, 4096, 1, 4096, 16},
      {257, 512, 1, 17, 3},     {130, 384, 1, 150, 200},  {100, 192, 90, 11, 8},     {2048, 7168, 16, 2048, 16},
      {72, 256, 6, 1300, 12},   {640, 512, 1, 0, 8},      {64, 128, 40, 3, 1},
  };
  // the library's own choices, then each path that can be forced
  const char *forced[][2] = {{nullptr, nullptr},          {"LORA4_BIG", "0"},         {"LORA4_BIG", "1"},
                             {"LORA4_FFN_DGRAD", "split"}, {"LORA4_FFN_DGRAD", "own"}, {"LORA4_FFN_ROWS", "4"},
                             {"LORA4_FFN_ROWS", "8"},      {"LORA4_FFN_ROWS", "1064"}, {"LORA4_FFN_ROWS", "1128"},
                             {"LORA4_FFN_ROWS", "1256"},   {"LORA4_FFN_ROWS", "2032"}, {"LORA4_FFN_ROWS", "2064"},
                             {"LORA4_FFN_ROWS", "2128"}};
  for (const auto &f : forced) {
    if (f[0]) setenv(f[0], f[1], 1);
    for (int fmt = LORA4_NF4; fmt <= LORA4_NVFP4; ++fmt)
      for (const Shape &s : shapes) {
        layer(fmt, s.N, s.K, s.E, s.M, s.r);
        feed_forward(fmt, s.N, s.K, s.E, s.M, s.r);
      }
    if (f[0]) unsetenv(f[0]);
  }
  norms();
  refusals();
  sizes();
  for (const auto &c : counts) std::printf("%s %d\n", c.first.c_str(), c.second);
  if (failures) return 1;
  std::printf("ok\n");
  return 0;
}
