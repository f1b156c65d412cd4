/* A HIP runtime that runs nothing: preloaded before libq8ta, it takes the place
 * of the runtime calls that the library makes and writes them down, so that
 * tests see on a CPU what a call would launch and allocate, and on which stream
 * it would wait.  Refuses what a launch cannot hold.  One line a call:
 *   launch <kernel> <grid x y z> <threads x y z> <stream>
 *   malloc <address> <bytes> <stream> | free <address> <stream>
 *   record <event> <stream> | wait <event> <stream> | query <event>
 */
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3_t;
enum { OK = 0, INVALID = 1, BAD_LAUNCH = 9, NOT_READY = 600 };

static char* text;
static size_t used, room;
static int last_error, capturing, pending, next_event = 1;
static uintptr_t next_address = (uintptr_t)1 << 32;

static void put(const char* fmt, ...) {
  if (room - used < 512) {
    room = room ? 2 * room : 1 << 20;
    text = realloc(text, room);
    if (!text) abort();
  }
  va_list ap;
  va_start(ap, fmt);
  used += (size_t)vsnprintf(text + used, room - used, fmt, ap);
  va_end(ap);
}

/* For the tests. */
const char* recorder_text(void) { return used ? text : ""; }
void recorder_clear(void) { used = 0; }
void recorder_capture(int on) { capturing = on; }   /* every stream is captured */
void recorder_pending(int on) { pending = on; }     /* events are not ready */

static struct { const void* fn; const char* name; } kernels[4096];
static int n_kernels;

void** __hipRegisterFatBinary(const void* data) { (void)data; return (void**)&kernels; }
void __hipUnregisterFatBinary(void** m) { (void)m; }
void __hipRegisterFunction(void** m, const void* fn, char* dev, const char* name, unsigned limit, void* tid,
                           void* bid, void* bdim, void* gdim, int* w) {
  (void)m; (void)dev; (void)limit; (void)tid; (void)bid; (void)bdim; (void)gdim; (void)w;
  if (n_kernels < 4096) { kernels[n_kernels].fn = fn; kernels[n_kernels++].name = name; }
}
void __hipRegisterVar(void** m, void* v, char* h, char* d, int e, size_t s, int c, int g) {
  (void)m; (void)v; (void)h; (void)d; (void)e; (void)s; (void)c; (void)g;
}
static dim3_t call_grid, call_block;
static size_t call_lds;
static void* call_stream;
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t lds, void* s) {
  call_grid = g; call_block = b; call_lds = lds; call_stream = s;
  return OK;
}
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* lds, void** s) {
  *g = call_grid; *b = call_block; *lds = call_lds; *s = call_stream;
  return OK;
}
int hipLaunchKernel(const void* fn, dim3_t g, dim3_t b, void** args, size_t lds, void* s) {
  (void)args; (void)lds;
  const char* name = "?";
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].fn == fn) name = kernels[i].name;
  put("launch %.200s %u %u %u %u %u %u %p\n", name, g.x, g.y, g.z, b.x, b.y, b.z, s);
  const uint64_t most = (uint64_t)1 << 32;
  if (!g.x || !g.y || !g.z || !b.x || !b.y || !b.z || (uint64_t)b.x * b.y * b.z > 1024 || (uint64_t)g.x * b.x >= most ||
      g.y > 65535 || g.z > 65535)
    return last_error = BAD_LAUNCH;
  return OK;
}
int hipGetLastError(void) { const int e = last_error; last_error = OK; return e; }
const char* hipGetErrorString(int e) { return e == BAD_LAUNCH ? "launch out of range" : "error"; }
int hipGetDevice(int* d) { *d = 0; return OK; }
int hipStreamIsCapturing(void* s, int* st) { (void)s; *st = capturing; return OK; }
int hipDeviceGetDefaultMemPool(void** p, int d) { (void)d; *p = &used; return OK; }
int hipMemPoolSetAttribute(void* p, int a, void* v) { (void)p; (void)a; (void)v; return OK; }
int hipMallocAsync(void** p, size_t bytes, void* s) {
  *p = (void*)next_address;
  next_address += (bytes + 4095) / 4096 * 4096 + 4096;
  put("malloc %p %zu %p\n", *p, bytes, s);
  return OK;
}
int hipFreeAsync(void* p, void* s) { put("free %p %p\n", p, s); return OK; }
int hipEventCreateWithFlags(void** e, unsigned f) { (void)f; *e = (void*)(uintptr_t)next_event++; return OK; }
int hipEventRecord(void* e, void* s) { put("record %p %p\n", e, s); return OK; }
int hipEventQuery(void* e) { put("query %p\n", e); return pending ? NOT_READY : OK; }
int hipStreamWaitEvent(void* s, void* e, unsigned f) { (void)f; put("wait %p %p\n", e, s); return OK; }
int hipFuncSetAttribute(const void* f, int a, int v) { (void)f; (void)a; (void)v; return OK; }
int hipGetSymbolAddress(void** p, const void* s) { (void)s; *p = (void*)next_address; return OK; }
