// Host-side check of the operators' device set-up: a CUDA call that fails once fails one call of theirs, not all that
// come later, and norms and draws do not depend on what only projections need.  The library's source is compiled in
// with the set-up's CUDA calls replaced; nothing runs on a GPU.  Exit status 1 on a violation.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdio>

static int fail_attribute = 0, fail_symbol = 0, fail_entry = 0, fail_function = 0;  // so many calls
static int calls = 0;
static cudaError_t once(int& left) {
  ++calls;
  return left > 0 ? (--left, cudaErrorStreamCaptureUnsupported) : cudaSuccess;
}
static cudaError_t fake_device(int* id) { return *id = 3, cudaSuccess; }
static cudaError_t fake_attribute(int* v) { return *v = 152, once(fail_attribute); }
static cudaError_t fake_symbol(void** p) { return *p = &calls, once(fail_symbol); }
static cudaError_t fake_entry(void** p, cudaDriverEntryPointQueryResult* found) {
  *p = &calls;
  *found = cudaDriverEntryPointSuccess;
  return once(fail_entry);
}
#define cudaGetDevice(id) fake_device(id)
#define cudaDeviceGetAttribute(v, which, id) fake_attribute(v)
#define cudaGetSymbolAddress(p, symbol) fake_symbol(p)
#define cudaGetDriverEntryPointByVersion(name, p, version, flags, found) fake_entry(p, found)
#define cudaFuncSetAttribute(f, which, v) once(fail_function)
#include "../request_token_sampling_gb300/csrc/strata_project.cu"

int strata::host_fail(int code, const char*, ...) { return code; }

int main() {
  int bad = 0;
  auto check = [&](bool ok, const char* what) {
    if (!ok) ++bad, std::printf("%s\n", what);
  };
  const Device* dev = nullptr;
  int id = -1;
  auto common = [&] { return current_device(&dev, &id, false); };
  auto projects = [&] { return current_device(&dev, &id, true); };
  fail_attribute = fail_symbol = 1;
  check(common() == STRATA_ECUDA, "the attribute's failure is told");
  check(common() == STRATA_ECUDA, "the symbol's failure is told");
  fail_entry = fail_function = 1;
  check(common() == STRATA_OK && id == 3 && dev->sms == 152 && dev->errors != nullptr, "norms and draws need no more");
  check(projects() == STRATA_ECUDA, "the entry point's failure is told");
  check(common() == STRATA_OK, "norms and draws go on");
  check(projects() == STRATA_ECUDA, "the function attribute's failure is told");
  check(projects() == STRATA_OK && dev->encode != nullptr, "projections go on");
  const int before = calls;
  check(common() == STRATA_OK && projects() == STRATA_OK && calls == before, "what is known is not asked again");
  std::printf("%d bad\n", bad);
  return bad == 0 ? 0 : 1;
}
