// Shared between the 8-bit matrices' sanitizer harness and its launch stand-ins.
#pragma once

namespace harness {
extern int q8_launches;
}
